// Verification of drafted codes: which of them stand, and the code that follows them.
//
// With p_i and q_i the model's and the draft's distributions at place i, draft x_i stands if u_i q_i(x_i) < p_i(x_i);
// behind the last that stands a code is drawn from max(p_i - q_i, 0) or, behind all drafts, from p_i.
//
// 64,000 borders lie in [0, 1), so the draw's probabilities and sums take 64 bits; a test has one border, so 32 bits
// settle all but about one in 1,000 (kDoubt), and those are taken again in 64.
//
// A cluster of up to 8 CTAs has a stream, a contiguous slice of the codes each.
//   scan: the rows' maxima and sums of exponentials in 32 bits (each thread's running maximum and sum), several rows at
//     a time, a job (a row, a part of the slice) to a warp.  With few streams all rows at once, as the chain
//     of barriers counts; with many a draft at a time, as the rows behind a refused one need not be read.
//   exact: the row that the draw is from (and the draft's) again, in 64 bits: the sums of the weights of each warp's
//     range; for max(p - q, 0) once more, now that both sums are known.
//   draw: the range, then the thread's share, then the code at which the running sum exceeds the target.
#include <algorithm>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {
namespace {

#define TOK_INLINE __attribute__((always_inline))

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxV = 1 << 18, kMaxK = 63;
constexpr int kRowsAtOnce = 2 * (int)kMaxK + 1;
constexpr float kLowest = -3.402823466e+38f;
// Relative: a lane adds up to 2^13 terms in fp32, each sum is within 2^13 2^-24 + 2^-20 (exponentials) < 2^-10.
constexpr double kDoubt = 1.0 / 512;

struct VerifyArgs {
    const void *logits, *draft;
    const int32_t *codes, *n_draft;
    const float *u, *temperature;
    float temperature_all;
    int32_t *out, *accepted;
    int64_t logits_batch, logits_row, draft_batch, draft_row;
    int K, V, slice; // codes per CTA
    int at_once;     // places scanned at once
};

// 16 bytes are N codes.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float one(const float *p) { return __ldg(p); }
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
        return bf16_lo(__ldg(reinterpret_cast<const unsigned short *>(p)));
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

__device__ __forceinline__ float exp2_approx(float x) // 2 ulp; 0 for -inf
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t ld_cluster64(const void *p, uint32_t rank)
{
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(mapa_shared(smem_addr(p), rank)) : "memory");
    return v;
}

// Order-preserving bits of a float (no NaN); -0 counts as 0.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// exp((x - top') / T) in 64 bits, top' so close to the row's largest logit that n0 below is whole (it falls out of every
// quotient): with y = 256 log2(e) x / T = n0 + k + f, k whole, 2^(k / 256) comes from a table and the exponent,
// 2^(f / 256) = 1 + f (c1 + f (c2 + f c3)): what is left out is below 2^-42 relative.  Weights below 2^-1000 of the largest,
// -inf and NaN are 0.  Of +inf as top, and where T is so small that y is no place in a table: 1 for top, 0 for all else.
constexpr int kTable = 256;
struct Weights {
    const double *table; // 2^(j / 256)
    double per_t, magic; // 256 log2(e) / T; 1.5 2^52 - n0
    float top, least;    // logits up to `least` have no weight, but for top
    bool only_top;
    __device__ __forceinline__ Weights(const double *table, float top, double T) : table(table), top(top)
    {
        per_t = kTable / 0.6931471805599453 / T;
        const double y = (double)top * per_t;
        only_top = !(fabs(y) < 1125899906842624.0); // 2^50
        magic = 6755399441055744.0 - rint(y);       // (a sum's low bits are its whole part)
        least = fmaxf((float)((double)top - 1000.0 * kTable / per_t), kLowest);
    }
    __device__ __forceinline__ double operator()(float x) const
    {
        constexpr double c1 = 0.6931471805599453 / kTable, c2 = c1 * c1 / 2, c3 = c2 * c1 / 3;
        if (__builtin_expect(only_top, 0))
            return x == top ? 1.0 : 0.0;
        const double d = (double)fmaxf(x, least), kd = fma(d, per_t, magic), f = fma(d, per_t, magic - kd);
        const int k = __double2loint(kd);
        const double t = table[k & (kTable - 1)], w = fma(t * f, fma(fma(c3, f, c2), f, c1), t);
        return x > least || x == top ? __hiloint2double(__double2hiint(w) + ((k >> 8) << 20), __double2loint(w)) : 0.0;
    }
};

struct Shared {
    double table[kTable];
    double sums[2][kWarps];         // of the warps' ranges
    uint64_t part[kRowsAtOnce][kWarps]; // of a row's parts: maximum and sum; greedy: the largest one's place
    uint64_t row[kRowsAtOnce];      // of this CTA's slice of each row
    float2 all[kRowsAtOnce];        // of the rows
    double range[kMaxCluster * kWarps];
    double warp[kWarps];
    int first, last;
};

__device__ __forceinline__ uint64_t as_bits(float2 x)
{
    return (uint64_t)__float_as_uint(x.y) << 32 | __float_as_uint(x.x);
}
__device__ __forceinline__ float2 as_pair(uint64_t x)
{
    return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs g, int C)
{
    constexpr int N = Vec<T>::N;
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int64_t b = blockIdx.x / C;
    const int begin = min(g.V, (int)rank * g.slice), n = min(g.slice, g.V - begin);
    const T *logits = static_cast<const T *>(g.logits) + b * g.logits_batch;
    const T *draft = g.draft ? static_cast<const T *>(g.draft) + b * g.draft_batch : nullptr;
    const int drafts = g.n_draft ? min(max(g.n_draft[b], 0), g.K) : g.K;
    const float *u = g.u + b * (g.K + 1);
    const int32_t *codes = g.codes + b * g.K;
    float temperature = g.temperature ? g.temperature[b] : g.temperature_all;
    const bool greedy = !(temperature > 0.0f);
    temperature = greedy ? 1.0f : fminf(temperature, 3.4e38f); // (an infinite one would turn infinite differences into NaN)
    const float per_t = fminf(fmaxf(1.4426950408889634f / temperature, 1e-37f), 3.4e38f); // a normal number
    if (tid < kTable)
        sh.table[tid] = exp2((double)tid / kTable);
    auto barrier = [&]() TOK_INLINE {
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
    };
    auto number = [](float v) TOK_INLINE { return v >= 0.0f ? fminf(v, 0.99999994f) : 0.0f; }; // in [0, 1); NaN: 0

    // A row's slice: `head` codes up to a 16-byte boundary, nv vectors, the rest.
    struct Slice {
        const T *p;
        int head, nv;
    };
    auto slice = [&](const T *row) TOK_INLINE {
        Slice s;
        s.p = row + begin;
        s.head = min(n, (int)((16 - ((uintptr_t)s.p & 15)) & 15) / (int)sizeof(T));
        s.nv = (n - s.head) / N;
        return s;
    };
    auto row_of = [&](int r, int i0) TOK_INLINE { // scanned rows: the model's of places i0 .., then the draft's
        const int places = min(g.at_once, drafts + 1 - i0);
        return r < places ? logits + (int64_t)(i0 + r) * g.logits_row : draft + (int64_t)(i0 + r - places) * g.draft_row;
    };

    // Maxima and sums of `rows` rows; greedy: the first of the largest instead.  A warp has its part of each row in
    // turn, the next kBatch x 32 vectors on their way while it works on the last.
    auto scan = [&](int rows, int i0) TOK_INLINE {
        constexpr int kBatch = 4;
        float m = kLowest, z = 0.0f;
        uint64_t best = 0;
        auto take = [&](const float *x, int count, int idx) TOK_INLINE {
            float top = x[0];
#pragma unroll
            for (int k = 1; k < N; ++k)
                if (k < count)
                    top = fmaxf(top, x[k]);
            if (greedy) {
                if (top >= m) { // (NaN: not)
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (k < count && x[k] >= kLowest) {
                            const uint64_t place = (uint64_t)order_key(x[k]) << 32 | (uint32_t)~(idx + k);
                            best = place > best ? place : best;
                        }
                    m = top;
                }
                return;
            }
            if (top > m) {
                z *= exp2_approx((m - top) * per_t);
                m = top;
            }
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (k < count)
                    z += exp2_approx((fmaxf(x[k], -INFINITY) - m) * per_t);
        };
        Slice s{};
        const uint4 *vec = nullptr;
        int v0 = 0, v1 = 0;
        auto part_of = [&](int r) TOK_INLINE { // this warp's vectors of row r
            s = slice(row_of(r, i0));
            const int per = (s.nv + kWarps - 1) / kWarps;
            v0 = min(s.nv, warp * per);
            v1 = min(s.nv, v0 + per);
            vec = reinterpret_cast<const uint4 *>(s.p + s.head);
        };
        uint4 next[kBatch];
        auto fetch = [&]() TOK_INLINE {
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (v0 + 32 * e + lane < v1)
                    next[e] = __ldg(vec + v0 + 32 * e + lane);
        };
        part_of(0);
        fetch();
        for (int r = 0; r < rows;) {
            uint4 v[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                v[e] = next[e];
            const Slice now = s;
            const int c0 = v0, c1 = v1;
            const bool last = c0 + 32 * kBatch >= c1; // of the row's part
            if (!last)
                v0 += 32 * kBatch;
            else if (r + 1 < rows)
                part_of(r + 1);
            if (!last || r + 1 < rows)
                fetch();
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
                if (c0 + 32 * e + lane < c1) {
                    float x[N];
                    Vec<T>::split(v[e], x);
                    take(x, N, begin + now.head + (c0 + 32 * e + lane) * N);
                }
            if (!last)
                continue;
            // The codes before the first vector (the first warp's) and behind the last one (the last warp's).
            const int odd0 = warp == 0 ? 0 : now.head + now.nv * N;
            const int odd1 = warp == 0 ? now.head : warp == kWarps - 1 ? n : odd0;
            for (int i = odd0 + lane; i < odd1; i += 32) {
                const float x = Vec<T>::one(now.p + i);
                take(&x, 1, begin + i);
            }
            if (greedy) {
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(~0u, best, o);
                    best = y > best ? y : best;
                }
            } else {
                float top = m;
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                z *= exp2_approx((m - top) * per_t);
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    z += __shfl_xor_sync(~0u, z, o);
                m = top;
            }
            if (lane == 0)
                sh.part[r][warp] = greedy ? best : as_bits(make_float2(m, z));
            m = kLowest;
            z = 0.0f;
            best = 0;
            ++r;
        }
        // One warp adds a row's parts up, then the CTAs' (in order).
        auto joined = [&](uint64_t mine) TOK_INLINE -> uint64_t { // lanes' parts, over kWarps lanes
            if (greedy) {
#pragma unroll
                for (int o = kWarps / 2; o; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(~0u, mine, o);
                    mine = y > mine ? y : mine;
                }
                return mine;
            }
            const float2 x = as_pair(mine);
            float top = x.x, sum;
#pragma unroll
            for (int o = kWarps / 2; o; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
            sum = x.y * exp2_approx((x.x - top) * per_t);
#pragma unroll
            for (int o = kWarps / 2; o; o >>= 1)
                sum += __shfl_xor_sync(~0u, sum, o);
            return as_bits(make_float2(top, sum));
        };
        const uint64_t none = greedy ? 0 : as_bits(make_float2(kLowest, 0.0f));
        __syncthreads();
        for (int r = warp; r < rows; r += kWarps) {
            const uint64_t x = joined(sh.part[r][lane % kWarps]);
            if (lane == 0)
                sh.row[r] = x;
        }
        barrier();
        for (int r = warp; r < rows; r += kWarps) {
            uint64_t x = sh.row[r];
            if (C > 1)
                x = joined(lane % kWarps < C ? ld_cluster64(&sh.row[r], lane % kWarps) : none);
            if (lane == 0) // greedy: the index's bits, inverted, and whether there is one
                sh.all[r] = greedy ? make_float2(__uint_as_float((uint32_t)x), x ? 1.0f : 0.0f) : as_pair(x);
        }
        barrier(); // (also: no CTA's rows are overwritten while another reads them)
    };
    auto weights_of = [&](float top) TOK_INLINE { return Weights(sh.table, top, (double)temperature); };
    // This warp's range [lo, hi) of the slice, in whole vectors of the row's.
    auto range_of = [&](int w, int &lo, int &hi) TOK_INLINE {
        const int per = ((n + kWarps - 1) / kWarps + N - 1) / N * N;
        lo = min(n, w * per);
        hi = min(n, lo + per);
    };
    // f(x of p, x of q, index) for this thread's codes of its warp's range; q may be null.
    auto codes_of = [&](const T *p, const T *q, int lo, int hi, auto &&f) TOK_INLINE {
        const bool vec = ((uintptr_t)(p + begin) & 15) == 0 && (!q || ((uintptr_t)(q + begin) & 15) == 0);
        const int nv = vec ? (hi - lo) / N : 0;
        const uint4 *pv = reinterpret_cast<const uint4 *>(p + begin + lo), *qv = reinterpret_cast<const uint4 *>(q + begin + lo);
        for (int i = lane; i < nv; i += 32) {
            float x[N], y[N];
            Vec<T>::split(__ldg(pv + i), x);
            if (q)
                Vec<T>::split(__ldg(qv + i), y);
#pragma unroll
            for (int k = 0; k < N; ++k)
                f(x[k], q ? y[k] : 0.0f, lo + i * N + k);
        }
        for (int i = lo + nv * N + lane; i < hi; i += 32)
            f(Vec<T>::one(p + begin + i), q ? Vec<T>::one(q + begin + i) : 0.0f, i);
    };
    auto warp_sum = [&](double v) TOK_INLINE {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(~0u, v, o);
        return v;
    };
    // The sums of all warps' ranges in all CTAs, in order, into sh.range; their sum.  Lane l of a warp has the
    // kEach from kEach l on.
    constexpr int kEach = kMaxCluster * kWarps / 32;
    auto gather = [&](int which) TOK_INLINE {
        barrier(); // every CTA has its own
        if (tid < kMaxCluster * kWarps) {
            const int c = tid / kWarps;
            sh.range[tid] = c >= C ? 0.0
                            : C > 1 ? __longlong_as_double((long long)ld_cluster64(&sh.sums[which][tid % kWarps], c))
                                    : sh.sums[which][tid];
        }
        barrier(); // (no CTA's sums are overwritten while another reads them)
        double v = 0.0;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            v += sh.range[lane * kEach + e];
        return warp_sum(v);
    };

    int place = 0; // the place that the code is drawn at
    bool refused = false;
    float2 p_row{}, q_row{};
    double zp = 0.0, zq = 0.0; // exact sums of the last row taken exactly
    // Exact sums of rows p and q (q may be null), without code `but` of the slice in p.
    auto exact = [&](const T *p, const T *q, int but) TOK_INLINE {
        const Weights wp = weights_of(p_row.x), wq = weights_of(q_row.x);
        int lo, hi;
        range_of(warp, lo, hi);
        double sp = 0.0, sq = 0.0;
        codes_of(p, q, lo, hi, [&](float x, float y, int i) TOK_INLINE {
            sp += i == but ? 0.0 : wp(x);
            if (q)
                sq += wq(y);
        });
        sp = warp_sum(sp);
        sq = warp_sum(sq);
        if (lane == 0) {
            sh.sums[0][warp] = sp;
            sh.sums[1][warp] = sq;
        }
        if (q)
            zq = gather(1);
        zp = gather(0); // (sh.range: those of p)
    };

    bool done = false;
    for (int i0 = 0; !done; i0 += g.at_once) {
        const int places = min(g.at_once, drafts + 1 - i0), tests = min(places, drafts - i0);
        scan(places + (draft ? tests : 0), i0);
        for (int k = 0; k < places; ++k) {
            place = i0 + k;
            p_row = sh.all[k];
            if (place == drafts) {
                done = true;
                break;
            }
            if (draft)
                q_row = sh.all[places + k];
            const int x = codes[place];
            const bool inside = x >= 0 && x < g.V;
            const double v = number(u[place]);
            bool stands;
            if (greedy)
                stands = inside && p_row.y != 0.0f && (int)~__float_as_uint(p_row.x) == x;
            else if (!inside)
                stands = false;
            else {
                const T *p = logits + (int64_t)place * g.logits_row, *q = draft ? draft + (int64_t)place * g.draft_row : nullptr;
                const Weights wp = weights_of(p_row.x), wq = weights_of(q_row.x);
                const double ep = wp(Vec<T>::one(p + x)), eq = q ? wq(Vec<T>::one(q + x)) : 1.0;
                // v eq / zq < ep / zp.  (eq is 0 where the draft's row has no code; the sums in 32 bits are of weights
                // relative to the largest logit.)
                double left = v * eq * ((double)p_row.y * wp(p_row.x));
                double right = ep * (q ? (double)q_row.y * wq(q_row.x) : 1.0);
                if (v * eq == 0.0 || ep == 0.0)
                    stands = ep > 0.0;
                else if (fabs(left - right) > kDoubt * right)
                    stands = left < right;
                else { // (sums of infinite logits are no numbers and come here, too)
                    exact(p, q, -1);
                    left = v * eq * zp;
                    right = ep * (q ? zq : 1.0);
                    stands = left < right;
                }
            }
            if (!stands) {
                refused = done = true;
                break;
            }
        }
    }

    // ---- The draw. ----
    if (rank == 0)
        for (int i = tid; i <= g.K; i += kThreads)
            if (i != place)
                g.out[b * (g.K + 1) + i] = i < place ? codes[i] : -1;
    if (rank == 0 && tid == 0)
        g.accepted[b] = place;
    auto emit = [&](int code) TOK_INLINE { g.out[b * (g.K + 1) + place] = code; };
    if (greedy) {
        if (rank == 0 && tid == 0)
            emit(p_row.y != 0.0f ? (int)~__float_as_uint(p_row.x) : -1);
        return; // (scan's last barrier was behind every read of another CTA's memory)
    }
    const T *p = logits + (int64_t)place * g.logits_row;
    const T *q = refused && draft ? draft + (int64_t)place * g.draft_row : nullptr;
    const Weights wp = weights_of(p_row.x), wq = weights_of(q_row.x);
    const int left_out = refused && !draft ? codes[place] : -1;
    int but = left_out >= begin && left_out < g.V ? left_out - begin : -1; // in this CTA's slice
    double rp = 1.0, rq = 0.0;
    bool minus = false;
    auto weight = [&](float x, float y, int i) TOK_INLINE {
        if (minus)
            return fmax(wp(x) * rp - wq(y) * rq, 0.0);
        return i == but ? 0.0 : wp(x);
    };
    exact(p, q, but);
    double total = zp;
    if (q && zp > 0.0 && zq > 0.0) {
        minus = true;
        rp = 1.0 / zp;
        rq = 1.0 / zq;
        int lo, hi;
        range_of(warp, lo, hi);
        double s = 0.0;
        codes_of(p, q, lo, hi, [&](float x, float y, int i) TOK_INLINE { s += weight(x, y, i); });
        s = warp_sum(s);
        if (lane == 0)
            sh.sums[0][warp] = s;
        total = gather(0);
    }
    if (total == 0.0 && refused) { // nothing is left: from p itself
        minus = false;
        but = -1;
        exact(p, nullptr, -1);
        total = zp;
    }
    if (total == 0.0) {
        if (rank == 0 && tid == 0)
            emit(-1);
        return;
    }
    double target = (double)number(u[g.K]) * total;
    // The range that the target lies in; the last with a weight where rounding leaves the target behind all.
    double mine = 0.0;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        mine += sh.range[lane * kEach + e];
    double run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(~0u, run, o);
        if (lane >= o)
            run += y;
    }
    run -= mine; // before this lane's
    int at = 0x7FFFFFFF, end = -1;
    double at_run = 0.0, end_run = 0.0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const double r = sh.range[lane * kEach + e];
        if (r > 0.0) {
            end = lane * kEach + e;
            end_run = run;
            if (at == 0x7FFFFFFF && run + r > target) {
                at = end;
                at_run = run;
            }
        }
        run += r;
    }
    const int first = (int)__reduce_min_sync(~0u, (unsigned)at), last = __reduce_max_sync(~0u, end);
    const int range = first != 0x7FFFFFFF ? first : last;
    target -= __shfl_sync(~0u, first != 0x7FFFFFFF ? at_run : end_run, range / kEach);
    if (range / kWarps != (int)rank)
        return;
    // The thread whose share of it the target lies in, then the code.
    int lo, hi;
    range_of(range % kWarps, lo, hi);
    const int per = (hi - lo + kThreads - 1) / kThreads, i0 = min(hi, lo + tid * per), i1 = min(hi, i0 + per);
    auto weight_at = [&](int i) TOK_INLINE {
        return weight(Vec<T>::one(p + begin + i), minus ? Vec<T>::one(q + begin + i) : 0.0f, i);
    };
    double share = 0.0;
    for (int i = i0; i < i1; ++i)
        share += weight_at(i);
    double upto = share;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(~0u, upto, o);
        if (lane >= o)
            upto += y;
    }
    if (lane == 31)
        sh.warp[warp] = upto;
    if (tid == 0) {
        sh.first = 0x7FFFFFFF;
        sh.last = -1;
    }
    __syncthreads();
    double before = upto - share;
    for (int w = 0; w < warp; ++w)
        before += sh.warp[w];
    if (share > 0.0) {
        if (before + share > target)
            atomicMin(&sh.first, tid);
        atomicMax(&sh.last, tid);
    }
    __syncthreads();
    if (tid != (sh.first != 0x7FFFFFFF ? sh.first : sh.last))
        return;
    int code = -1;
    for (int i = i0; i < i1; ++i) {
        const double w = weight_at(i);
        before += w;
        if (w > 0.0) {
            code = begin + i;
            if (before > target)
                break;
        }
    }
    emit(code);
}

template <typename T> tok_status launch(VerifyArgs g, int64_t B, cudaStream_t stream)
{
    constexpr int N = Vec<T>::N;
    auto slice_of = [&](int c) { return ((g.V + c - 1) / c + N - 1) / N * N; };
    // CTAs per stream: as many as are resident at a time, two to an SM.
    const int64_t fit = std::max<int64_t>(1, 2 * 148 / B), need = std::max<int64_t>(1, g.V / (2 * kThreads));
    const int C = (int)std::min(std::min<int64_t>(kMaxCluster, fit), need);
    g.slice = slice_of(C);
    g.at_once = B * C <= 2 * 148 ? g.K + 1 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<T>, g, C);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }
    return launch_status();
}

} // namespace
} // namespace tok

extern "C" tok_status tok_verify_codes(const void *logits, const void *draft_logits, tok_dtype dtype,
                                       const int32_t *codes, const float *u, const int32_t *n_draft,
                                       const float *temperature, float temperature_all, int32_t *out,
                                       int32_t *accepted, int64_t B, int64_t K, int64_t V, int64_t logits_batch,
                                       int64_t logits_row, int64_t draft_batch, int64_t draft_row,
                                       cudaStream_t stream)
{
    using namespace tok;
    if (dtype != TOK_F32 && dtype != TOK_BF16)
        return TOK_ERR_DTYPE;
    const int64_t size = dtype == TOK_F32 ? 4 : 2;
    constexpr int64_t kStride = (int64_t)1 << 40;
    if (B < 0 || B > ((int64_t)1 << 20) || K < 0 || K > kMaxK || V < 1 || V > kMaxV)
        return TOK_ERR_SHAPE;
    if (K == 0)
        draft_logits = nullptr, codes = nullptr; // there is nothing of them
    for (int64_t s : {B > 1 ? logits_batch : 0, K > 0 ? logits_row : 0, draft_logits && B > 1 ? draft_batch : 0,
                      draft_logits && K > 1 ? draft_row : 0})
        if (s < 0 || s >= kStride)
            return TOK_ERR_SHAPE;
    if (B == 0)
        return TOK_OK;
    if (!logits || !u || !out || !accepted || (K > 0 && !codes))
        return TOK_ERR_NULL;
    if (!aligned(logits, size) || !aligned(draft_logits, size) || !aligned(codes, 4) || !aligned(u, 4) ||
        !aligned(n_draft, 4) || !aligned(temperature, 4) || !aligned(out, 4) || !aligned(accepted, 4))
        return TOK_ERR_ALIGN;
    struct Range {
        const void *p;
        int64_t bytes;
    };
    const Range ins[] = {{logits, ((B - 1) * logits_batch + K * logits_row + V) * size},
                         {draft_logits, ((B - 1) * draft_batch + (K - 1) * draft_row + V) * size},
                         {codes, 4 * B * K},
                         {u, 4 * B * (K + 1)},
                         {n_draft, 4 * B},
                         {temperature, 4 * B}};
    const Range outs[] = {{out, 4 * B * (K + 1)}, {accepted, 4 * B}};
    for (const Range &o : outs)
        for (const Range &i : ins)
            if (i.p && overlaps(i.p, i.bytes, o.p, o.bytes))
                return TOK_ERR_ALIAS;
    if (overlaps(out, 4 * B * (K + 1), accepted, 4 * B))
        return TOK_ERR_ALIAS;
    VerifyArgs g{};
    g.logits = logits;
    g.draft = draft_logits;
    g.codes = codes;
    g.n_draft = n_draft;
    g.u = u;
    g.temperature = temperature;
    g.temperature_all = temperature_all;
    g.out = out;
    g.accepted = accepted;
    g.logits_batch = logits_batch;
    g.logits_row = logits_row;
    g.draft_batch = draft_batch;
    g.draft_row = draft_row;
    g.K = (int)K;
    g.V = (int)V;
    return dtype == TOK_F32 ? launch<float>(g, B, stream) : launch<__nv_bfloat16>(g, B, stream);
}
