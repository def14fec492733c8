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
// A cluster of C CTAs holds one row in shared memory, a contiguous slice in each: the row
// is read from HBM once.  Ranks come from a histogram (counts and weights over 1024 bins
// of x), then from the few tokens of the bin in which the limit lies, sorted outright; a
// bin with more than kCap tokens is first narrowed on the bits of x, to a single value if
// need be, whose ties are then counted in index order.
#include <algorithm>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 1024;          // one per thread
constexpr int kCap = 1024;           // tokens sorted outright
constexpr int kSeg = 256;            // tokens per segment of the final running sum
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxV = 1 << 18;
constexpr double kOne = 17592186044416.0; // 2^44
constexpr float kReach = 31.25f;     // exp(-31.25) 2^44 < 1/2: no weight beyond

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
    int V, slice, segs; // tokens per CTA (a multiple of kSeg), segments per CTA
    int vec;            // rows may be read 16 bytes at a time
};

// Order-preserving bits of a float (no NaN, no -0 here).
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float clean(float x) { return isnan(x) ? -INFINITY : x + 0.0f; } // -0 counts as 0

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

struct Cut { // kept: key > .key, or key == .key and index <= .idx
    uint32_t key;
    int idx;
};

struct Shared {
    uint64_t wsum[kBins];   // weight histogram: lo in [0, kBins), hi after it, as 32-bit words
    uint32_t cnt[kBins];
    uint64_t list_w[kCap];
    uint32_t list_key[kCap], sort_key[kCap];
    int list_idx[kCap], sort_idx[kCap];
    uint64_t warp64[kWarps];
    uint64_t found_before;
    uint64_t cta_total;
    uint32_t warp32[kWarps];
    uint32_t pub[4]; // this CTA's largest and smallest key, list length, tie count
    uint32_t found_bin, found_cnt, res_key, res_idx;
    uint64_t found_mass;
};

template <typename T> struct Row1; // raw values in shared memory
template <> struct Row1<float> {
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <> struct Row1<__nv_bfloat16> {
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p)
    {
        return bf16_lo(*reinterpret_cast<const unsigned short *>(p));
    }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// Inclusive scan over the block's threads; *total gets the sum.  All threads.
__device__ uint64_t block_scan(uint64_t v, uint64_t *warp, uint64_t *total)
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
    if (w == 0) {
        uint64_t s = warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(~0u, s, o);
            if (lane >= o)
                s += x;
        }
        warp[lane] = s;
    }
    __syncthreads();
    *total = warp[kWarps - 1];
    return v + (w ? warp[w - 1] : 0);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs g, int C)
{
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    uint64_t *seg = reinterpret_cast<uint64_t *>(smem + sizeof(Shared));
    T *vals = reinterpret_cast<T *>(smem + sizeof(Shared) + 8 * (size_t)g.segs);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const int begin = min(g.V, (int)rank * g.slice), n = min(g.slice, g.V - begin);
    auto sync_all = [&] {
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
    };

    float T1 = g.temperature ? g.temperature[row] : g.temperature_all;
    const float top_p = g.top_p ? g.top_p[row] : g.top_p_all;
    float min_p = g.min_p ? g.min_p[row] : g.min_p_all;
    min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
    int top_k = g.top_k ? g.top_k[row] : g.top_k_all;
    if (!(T1 > 0.0f) || top_p <= 0.0f) { // greedy; or the nucleus is the largest token alone
        top_k = 1;
        T1 = T1 > 0.0f ? T1 : 1.0f;
    }
    T1 = fminf(T1, 3.4e38f); // (an infinite one would turn -inf logits into NaN)
    const double inv_t = 1.0 / (double)T1;

    // The slice into shared memory, its largest value and its smallest finite one.
    uint32_t kmax = 0, kmin = ~0u;
    {
        const T *src = static_cast<const T *>(g.logits) + row * g.row_stride + begin;
        constexpr int N = 16 / sizeof(T);
        const uint32_t lowest = order_key(-INFINITY);
        auto put = [&](int i, float x) {
            x = clean(x);
            vals[i] = Row1<T>::put(x);
            const uint32_t k = order_key(x);
            kmax = max(kmax, k);
            if (k != lowest)
                kmin = min(kmin, k);
        };
        int i0 = 0;
        if (g.vec) {
            i0 = n / N * N;
            for (int i = tid * N; i < i0; i += kThreads * N) {
                float v[N];
                Row<T, N, true>::load(src + i, v);
#pragma unroll
                for (int k = 0; k < N; ++k)
                    put(i + k, v[k]);
            }
        }
        for (int i = i0 + tid; i < n; i += kThreads)
            put(i, Row1<T>::get(src + i));
    }
    kmax = __reduce_max_sync(~0u, kmax);
    kmin = __reduce_min_sync(~0u, kmin);
    if (lane == 0) {
        sh.warp32[warp] = kmax;
        reinterpret_cast<uint32_t *>(sh.warp64)[warp] = kmin;
    }
    __syncthreads();
    if (tid < 32) {
        const uint32_t a = __reduce_max_sync(~0u, sh.warp32[lane]);
        const uint32_t b = __reduce_min_sync(~0u, reinterpret_cast<uint32_t *>(sh.warp64)[lane]);
        if (lane == 0) {
            sh.pub[0] = a;
            sh.pub[1] = b;
        }
    }
    sync_all();
    for (int c = 0; c < C; ++c) {
        kmax = max(kmax, C > 1 ? ld_cluster(smem_addr(&sh.pub[0]), c) : sh.pub[0]);
        kmin = min(kmin, C > 1 ? ld_cluster(smem_addr(&sh.pub[1]), c) : sh.pub[1]);
    }
    auto value = [](uint32_t key) { return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key); };
    const float xmax = value(kmax);
    if (xmax == -INFINITY) { // nothing to draw from
        if (rank == 0 && tid == 0) {
            g.idx[row] = -1;
            if (g.logprob)
                g.logprob[row] = -INFINITY;
        }
        sync_all(); // no CTA leaves while another reads its shared memory
        return;
    }
    auto z_of = [&](float x) { return x == xmax ? 0.0 : ((double)x - (double)xmax) * inv_t; };
    auto weight = [&](double z) -> uint64_t { return z < -31.25 ? 0ull : (uint64_t)__double2ull_rn(exp(z) * kOne); };

    // ---- Ranks: the last token kept by top-k, then by top-p. ----
    Cut cut{0u, 0x7FFFFFFF};
    const bool by_k = top_k > 0 && top_k < g.V, by_p = top_p < 1.0f && top_k != 1;
    if (by_k || by_p) {
        uint32_t *lo = reinterpret_cast<uint32_t *>(sh.wsum), *hi = lo + kBins;
        // Bins of equal width over the values that can have a weight.
        const float span = fminf(kReach * T1, xmax - value(kmin));
        const float per = span > 0.0f ? (float)kBins / span : 0.0f;
        const uint32_t lowest = order_key(-INFINITY);

        // Histogram of the tokens with klo <= key <= khi over 1024 bins, the highest values in bin 0:
        // of x on the first pass (shift < 0), of the key's bits after it.  Every CTA then adds up all
        // slices' bins; thread j returns with bin j's totals.
        auto histogram = [&](uint32_t klo, uint32_t khi, int shift, uint64_t &c_out, uint64_t &w_out) {
            sh.cnt[tid] = 0;
            lo[tid] = hi[tid] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const float x = Row1<T>::get(vals + i);
                const uint32_t k = order_key(x);
                if (k == lowest || k < klo || k > khi)
                    continue;
                int b;
                if (shift < 0) {
                    const float d = x == xmax ? 0.0f : (xmax - x) * per;
                    b = min(kBins - 1, (int)d);
                } else
                    b = (int)((khi - k) >> shift);
                atomicAdd(&sh.cnt[b], 1u);
                if (by_p) {
                    const uint64_t w = weight(z_of(x));
                    const uint32_t wl = (uint32_t)w, old = atomicAdd(&lo[b], wl);
                    const uint32_t wh = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
                    if (wh)
                        atomicAdd(&hi[b], wh);
                }
            }
            sync_all();
            c_out = w_out = 0;
            for (int c = 0; c < C; ++c) {
                if (C > 1) {
                    c_out += ld_cluster(smem_addr(&sh.cnt[tid]), c);
                    if (by_p)
                        w_out += (uint64_t)ld_cluster(smem_addr(&lo[tid]), c) +
                                 ((uint64_t)ld_cluster(smem_addr(&hi[tid]), c) << 32);
                } else {
                    c_out += sh.cnt[tid];
                    w_out += (uint64_t)lo[tid] + ((uint64_t)hi[tid] << 32);
                }
            }
            sync_all(); // the bins may be cleared again
        };

        // The tokens of [klo, khi] (at most kCap) of all slices, sorted by falling key, then index:
        // sort_key / sort_idx / list_w (weights); returns their number.
        auto sorted_list = [&](uint32_t klo, uint32_t khi) -> int {
            if (tid == 0)
                sh.pub[2] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const uint32_t k = order_key(Row1<T>::get(vals + i));
                if (k >= klo && k <= khi) {
                    const uint32_t at = atomicAdd(&sh.pub[2], 1u);
                    if (at < (uint32_t)kCap) {
                        sh.list_key[at] = k;
                        sh.list_idx[at] = begin + i;
                    }
                }
            }
            sync_all();
            int total = 0;
            uint32_t my_key = 0;
            int my_idx = 0;
            for (int c = 0; c < C; ++c) {
                const int m = (int)(C > 1 ? ld_cluster(smem_addr(&sh.pub[2]), c) : sh.pub[2]);
                if (tid >= total && tid < total + m) {
                    my_key = C > 1 ? ld_cluster(smem_addr(&sh.list_key[tid - total]), c) : sh.list_key[tid - total];
                    my_idx = (int)(C > 1 ? ld_cluster(smem_addr(&sh.list_idx[tid - total]), c)
                                         : (uint32_t)sh.list_idx[tid - total]);
                }
                total += m;
            }
            sync_all();
            if (tid < total) { // all slices' tokens, in any order
                sh.list_key[tid] = my_key;
                sh.list_idx[tid] = my_idx;
            }
            __syncthreads();
            if (tid < total) {
                int r = 0;
                for (int j = 0; j < total; ++j) {
                    const uint32_t k = sh.list_key[j];
                    r += k > my_key || (k == my_key && sh.list_idx[j] < my_idx);
                }
                sh.sort_key[r] = my_key;
                sh.sort_idx[r] = my_idx;
                sh.list_w[r] = weight(z_of(value(my_key)));
            }
            __syncthreads();
            return total;
        };

        // Index of the m-th (from 1) token with this very key, in index order.
        auto nth_tie = [&](uint32_t key, uint32_t m) -> int {
            const int per_thread = (n + kThreads - 1) / kThreads, i0 = min(n, tid * per_thread),
                      i1 = min(n, i0 + per_thread);
            uint64_t c = 0, total;
            for (int i = i0; i < i1; ++i)
                c += order_key(Row1<T>::get(vals + i)) == key;
            uint64_t incl = block_scan(c, sh.warp64, &total);
            if (tid == 0) {
                sh.pub[3] = (uint32_t)total;
                sh.res_idx = 0;
            }
            sync_all();
            uint64_t before = 0;
            for (uint32_t r = 0; r < rank; ++r)
                before += ld_cluster(smem_addr(&sh.pub[3]), r);
            incl += before;
            if (c && incl >= m && incl - c < m) {
                uint64_t at = incl - c;
                for (int i = i0; i < i1; ++i)
                    if (order_key(Row1<T>::get(vals + i)) == key && ++at == m)
                        sh.res_idx = (uint32_t)(begin + i) + 1;
            }
            sync_all();
            uint32_t idx = 0; // the one slice that has it wrote index + 1
            for (int c2 = 0; c2 < C; ++c2)
                idx = max(idx, C > 1 ? ld_cluster(smem_addr(&sh.res_idx), c2) : sh.res_idx);
            sync_all();
            return (int)idx - 1;
        };

        // The key range of the tokens of bin b of the first histogram.
        auto range_of_bin = [&](int b, uint32_t &klo, uint32_t &khi) {
            uint32_t a = 0, z = ~0u;
            for (int i = tid; i < n; i += kThreads) {
                const float x = Row1<T>::get(vals + i);
                const uint32_t k = order_key(x);
                const float d = x == xmax ? 0.0f : (xmax - x) * per;
                if (k != lowest && min(kBins - 1, (int)d) == b) {
                    a = max(a, k);
                    z = min(z, k);
                }
            }
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
            sync_all();
            khi = 0;
            klo = ~0u;
            for (int c = 0; c < C; ++c) {
                khi = max(khi, C > 1 ? ld_cluster(smem_addr(&sh.pub[0]), c) : sh.pub[0]);
                klo = min(klo, C > 1 ? ld_cluster(smem_addr(&sh.pub[1]), c) : sh.pub[1]);
            }
            sync_all();
        };

        uint64_t cnt0, mass0, total_cnt, total_mass;
        histogram(0u, ~0u, -1, cnt0, mass0);
        const uint64_t cnt0_incl = block_scan(cnt0, sh.warp64, &total_cnt);
        const uint64_t mass0_incl = block_scan(mass0, sh.warp64, &total_mass);

        // One limit: by count (the `want`-th token) or by weight (the last token before which less
        // than `limit` lies).  Tokens past `cut` do not count.
        auto find = [&](bool count, uint64_t want, double limit) {
            uint64_t before_c = 0, before_w = 0;
            uint32_t klo = 0, khi = 0, m = 0;
            {
                const bool here = count ? cnt0_incl >= want && cnt0_incl - cnt0 < want
                                        : (double)mass0_incl >= limit && (double)(mass0_incl - mass0) < limit;
                __syncthreads();
                if (here) {
                    sh.found_bin = (uint32_t)tid;
                    sh.found_cnt = (uint32_t)cnt0;
                    sh.found_before = cnt0_incl - cnt0;
                    sh.found_mass = mass0_incl - mass0;
                }
                __syncthreads();
                before_c = sh.found_before;
                before_w = sh.found_mass;
                m = sh.found_cnt;
                range_of_bin((int)sh.found_bin, klo, khi);
            }
            while (m > (uint32_t)kCap && klo < khi) { // narrow the range on the key's bits
                int shift = 0;
                while (((khi - klo) >> shift) >= (uint32_t)kBins)
                    ++shift;
                uint64_t c, w, tc, tw;
                histogram(klo, khi, shift, c, w);
                const uint64_t ci = block_scan(c, sh.warp64, &tc), wi = block_scan(w, sh.warp64, &tw);
                const bool here = count ? before_c + ci >= want && before_c + ci - c < want
                                        : (double)(before_w + wi) >= limit && (double)(before_w + wi - w) < limit;
                __syncthreads();
                if (here) {
                    sh.found_bin = (uint32_t)tid;
                    sh.found_cnt = (uint32_t)c;
                    sh.found_before = before_c + ci - c;
                    sh.found_mass = before_w + wi - w;
                }
                __syncthreads();
                before_c = sh.found_before;
                before_w = sh.found_mass;
                m = sh.found_cnt;
                const uint32_t b = sh.found_bin, top = khi;
                khi = top - (b << shift);
                klo = max(klo, shift ? khi - ((1u << shift) - 1) : khi);
            }
            uint64_t kept_mass = 0; // weight of the tokens up to the limit
            if (m <= (uint32_t)kCap) {
                const int total = sorted_list(klo, khi);
                const bool live = tid < total;
                uint64_t tw;
                const uint64_t w = live ? sh.list_w[tid] : 0, wi = block_scan(w, sh.warp64, &tw);
                const bool in_cut = live && (sh.sort_key[tid] > cut.key ||
                                             (sh.sort_key[tid] == cut.key && sh.sort_idx[tid] <= cut.idx));
                const bool keep = in_cut && (count ? before_c + tid < want : (double)(before_w + wi - w) < limit);
                const int kept = __syncthreads_count(keep); // a prefix of the list
                if (kept > 0 && tid == kept - 1) {
                    sh.res_key = sh.sort_key[tid];
                    sh.res_idx = (uint32_t)sh.sort_idx[tid];
                    sh.found_mass = before_w + wi;
                }
                __syncthreads();
                if (kept > 0) {
                    cut.key = sh.res_key;
                    cut.idx = (int)sh.res_idx;
                    kept_mass = sh.found_mass;
                }
                __syncthreads();
            } else { // one value, more than kCap times: its first ties in index order
                const uint64_t w = weight(z_of(value(klo)));
                uint64_t take = m;
                if (count)
                    take = want - before_c;
                else if (w) { // the most ties j with before + (j - 1) w < limit
                    const double room = ceil((limit - (double)before_w) / (double)w);
                    take = room < 1.0 ? 1 : room < (double)m ? (uint64_t)room : m;
                }
                const int idx = nth_tie(klo, (uint32_t)take);
                if (klo != cut.key || idx < cut.idx)
                    cut = Cut{klo, idx};
                kept_mass = before_w + take * w;
            }
            return kept_mass;
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

    // ---- Running sum of the kept weights, by segments of kSeg tokens in index order. ----
    auto kept_weight = [&](int i) -> uint64_t { // token i of this slice
        const float x = Row1<T>::get(vals + i);
        const uint32_t k = order_key(x);
        if (k < cut.key || (k == cut.key && begin + i > cut.idx))
            return 0;
        const double z = z_of(x);
        if (z < -31.25)
            return 0;
        const double e = exp(z);
        return e >= (double)min_p ? (uint64_t)__double2ull_rn(e * kOne) : 0ull;
    };
    const int segs = (n + kSeg - 1) / kSeg;
    uint64_t mine = 0;
    for (int s = warp; s < segs; s += kWarps) {
        uint64_t w = 0;
#pragma unroll
        for (int k = 0; k < kSeg / 32; ++k) {
            const int i = s * kSeg + k * 32 + lane;
            if (i < n)
                w += kept_weight(i);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
            w += __shfl_xor_sync(~0u, w, o);
        if (lane == 0)
            seg[s] = w;
        mine += w;
    }
    uint64_t all;
    block_scan(lane == 0 ? mine : 0, sh.warp64, &all);
    if (tid == 0)
        sh.cta_total = all;
    sync_all();
    uint64_t before = 0, total = 0, own = 0;
    for (int c = 0; c < C; ++c) {
        const uint64_t t = C > 1 ? ld_cluster64(smem_addr(&sh.cta_total), c) : sh.cta_total;
        if (c < (int)rank)
            before += t;
        if (c == (int)rank)
            own = t;
        total += t;
    }
    // The first token at which the running sum exceeds u * total: an integer sum exceeds it
    // exactly when it exceeds its floor.
    const double ut = fmin(fmax((double)g.u[row], 0.0), 1.0) * (double)total;
    const uint64_t target = min((uint64_t)ut, total - 1);
    if (target >= before && target < before + own && warp == 0) {
        uint64_t run = before;
        int s = 0;
        for (int s0 = 0; s0 < segs; s0 += 32) { // the segment
            uint64_t v = s0 + lane < segs ? seg[s0 + lane] : 0;
            const uint64_t one = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t x = __shfl_up_sync(~0u, v, o);
                if (lane >= o)
                    v += x;
            }
            const uint32_t hit = __ballot_sync(~0u, run + v > target);
            if (hit) {
                const int l = __ffs(hit) - 1;
                s = s0 + l;
                run += __shfl_sync(~0u, v - one, l);
                break;
            }
            run += __shfl_sync(~0u, v, 31);
        }
        for (int k = 0; k < kSeg / 32; ++k) { // the token
            const int i = s * kSeg + k * 32 + lane;
            uint64_t v = i < n ? kept_weight(i) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t x = __shfl_up_sync(~0u, v, o);
                if (lane >= o)
                    v += x;
            }
            const uint32_t hit = __ballot_sync(~0u, run + v > target);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    g.idx[row] = begin + i;
                    if (g.logprob)
                        g.logprob[row] = (float)(z_of(Row1<T>::get(vals + i)) - log((double)total / kOne));
                }
                break;
            }
            run += __shfl_sync(~0u, v, 31);
        }
    }
    sync_all(); // no CTA leaves while another reads its shared memory
}

template <typename T> tok_status launch(const SampleArgs &g, int C, int64_t R, size_t smem, cudaStream_t stream)
{
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

    // CTAs per row: as few as hold the row in shared memory, more (up to 8) while the GPU
    // has idle SMs.
    auto slice_of = [&](int c) { return ((V + c - 1) / c + kSeg - 1) / kSeg * kSeg; };
    auto bytes_of = [&](int c) {
        return sizeof(Shared) + 8 * (size_t)(slice_of(c) / kSeg) + (size_t)(slice_of(c) * size);
    };
    int C = 1;
    while (C < kMaxCluster && (bytes_of(C) > 225 * 1024 || (R * C * 2 <= 148 && slice_of(C) > 2 * kThreads)))
        C *= 2;
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
    g.slice = (int)slice_of(C);
    g.segs = g.slice / kSeg;
    g.vec = aligned(logits, 16) && (R == 1 || row_stride * size % 16 == 0);
    return dtype == TOK_F32 ? launch<float>(g, C, R, bytes_of(C), stream)
                            : launch<__nv_bfloat16>(g, C, R, bytes_of(C), stream);
}
