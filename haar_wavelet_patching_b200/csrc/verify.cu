// Verification of drafted codes: which of them stand, and the code that follows them.
//
// With p_i and q_i the model's and the draft's distributions at place i, draft x_i stands if u_i q_i(x_i) < p_i(x_i);
// behind the last that stands a code is drawn from max(p_i - q_i, 0) or, behind all drafts, from p_i.
//
// As many borders as codes lie in [0, 1), so the draw's weights and sums take more than 32 bits (Weights); a test has
// one border, so that 32 bits settle all but about one in 1,000 (kDoubt), and those are taken again.
//
// scan_kernel: the maxima and sums of exponentials of all rows that a draft or the code behind the drafts may need,
//   in 32 bits (each thread's running maximum and sum), a part of a row to a CTA: one pass.
// verify_kernel, launched early: a cluster of up to 8 CTAs has a stream, a contiguous slice of the codes each.  All
//   tests at once; then the row that the draw is from, and the draft's, by Weights: the sums of the weights of each
//   warp's range, for max(p - q, 0) once more, now that both sums are known; the range, then the thread's share, then
//   the code at which the running sum exceeds the target.
// Measured, 64,000 codes: 96 streams of up to 6 drafts, fp32, 90 us: the scan 32 (172 MB, 5.4 TB/s), then two passes of
// 12 million weights, bound by the latency of a weight's chain at 24 warps an SM; 4 streams of 4 drafts, bf16, 22 us,
// a chain of short steps.
#include <algorithm>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {
namespace {

#define TOK_INLINE __attribute__((always_inline))

constexpr int kThreads = 256, kCtas = 3, kWarps = kThreads / 32; // (kCtas to an SM in verify_kernel)
constexpr int kMaxThreads = kCtas * kThreads, kMaxWarps = kMaxThreads / 32; // of verify_kernel's CTAs with few streams
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxV = 1 << 18, kMaxK = 63;
constexpr int kMaxRows = 2 * (int)kMaxK + 1;
constexpr int kCodes = 2;     // of a lane at a time in a pass (4 spill: 24.5 us for 22.5 with 4 streams)
constexpr int kMaxParts = 16; // of a row in the scan
constexpr float kLowest = -3.402823466e+38f;
// Relative: a thread adds up to 2^7 terms in fp32 and exponentials are within 2^-15 (the rounding of arguments up to
// 126), so a sum is within 2^-14 and a test within four times that.
constexpr double kDoubt = 1.0 / 512;

struct VerifyArgs {
    const void *logits, *draft;
    const int32_t *codes, *n_draft;
    const float *u, *temperature;
    float temperature_all;
    int32_t *out, *accepted;
    int64_t logits_batch, logits_row, draft_batch, draft_row;
    int K, V, slice; // codes per CTA
    int parts, part; // of a row in the scan; codes of a part
    uint64_t *stats; // [B][2 K + 1][parts], the model's rows, then the draft's: maximum and sum; greedy: the largest's place
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

// exp((x - top) / T), top the row's largest logit, but for a factor of the row (`unit`), within 2^-33 and as a 64-bit
// number, with most of its steps in 32 bits.  With x - base exact, its product with 1024 log2(e) / T (two 32-bit
// numbers, lo the rest of hi) is k + f, k whole; 2^(k / 1024) comes from a table and the exponent, 2^(f / 1024) - 1 =
// f (c1 + f c2) (|f c1| < 2^-11: the cubic term is below 2^-36, the rounding of f and of the polynomial below 2^-34).
// base is 0 up to |top| / T of 2000: logits that count are then below 2700 T and k below 2^22.  Above that it is top:
// logits that count differ from top by less than half of it, so that the difference is exact.  Such errors of 64,000
// weights do not add up to what would move a draw; one weight by itself is taken with exact_weight.  Weights below
// 2^-1000 of the largest, -inf and NaN are 0.  Of +inf as top, or with a temperature next to 0, only top counts.
constexpr int kTable = 1024;
struct Weights {
    const double *table; // 2^(j / 1024)
    double per_t;        // 1024 log2(e) / T
    double far;          // logits that much below the largest have no weight
    float hi, lo;
    bool only_top;
    __device__ __forceinline__ Weights(const double *table, float T) : table(table)
    {
        per_t = kTable / 0.6931471805599453 / (double)T;
        far = 1000.0 * kTable / per_t;
        only_top = !(per_t < 1e30);
        hi = (float)per_t;
        lo = (float)(per_t - (double)hi);
    }
    struct Row {
        float top, least; // logits from `least` on have a weight
        float base, cap, hi, lo;
        int k;
        bool only_top;
    };
    __device__ __forceinline__ Row row(float top) const
    {
        Row r;
        r.top = top;
        r.only_top = only_top || top == INFINITY;
        r.least = r.only_top ? top : fmaxf((float)((double)top - far), kLowest);
        r.cap = fminf(top, -kLowest);
        r.base = r.only_top || fabs((double)top * per_t) > 2000.0 * kTable / 0.6931471805599453 ? r.cap : 0.0f;
        r.hi = r.only_top ? 0.0f : hi;
        r.lo = r.only_top ? 0.0f : lo;
        r.k = 0x4B400000 + (r.base == 0.0f ? __double2int_rn((double)top * per_t) : 0);
        return r;
    }
    // What all weights of a row are divided by here.
    __device__ __forceinline__ double unit(const Row &r) const
    {
        return r.base == 0.0f && !r.only_top ? exp2(((double)(r.k - 0x4B400000) - (double)r.top * per_t) / kTable) : 1.0;
    }
    // (No branch, so that several weights are under way at a time.)
    __device__ __forceinline__ double operator()(const Row &r, float x) const
    {
        constexpr float c1 = (float)(0.6931471805599453 / kTable), c2 = c1 * c1 / 2;
        const float d = fminf(x, r.cap) - r.base;
        const float m = fmaf(d, r.hi, 12582912.0f); // (1.5 2^23: a sum's low bits are its whole part)
        const float f = fmaf(d, r.lo, fmaf(d, r.hi, 12582912.0f - m));
        const int k = __float_as_int(m) - r.k;
        const double t = table[k & (kTable - 1)], w = fma(t, (double)(f * fmaf(f, c2, c1)), t);
        const bool some = x >= r.least;
        return __hiloint2double(some ? __double2hiint(w) + ((k << 10) & 0xFFF00000) : 0, some ? __double2loint(w) : 0);
    }
};
// (By itself: it is long, and the code that all CTAs run through has to be short, as each fetches it once.)
__device__ __noinline__ double exact_weight(float top, float least, bool only_top, float x, float T)
{
    return !(x >= least) ? 0.0 : only_top ? 1.0 : exp(((double)x - (double)top) / (double)T);
}

struct Shared {
    double table[kTable], steps[2][32]; // 2^(j / 1024); 2^(j / 32), 2^(j / 1024)
    double sums[2][2][kMaxWarps];          // of the warps' ranges in p and in q, two passes' in turn
    float2 all[kMaxRows];               // of the rows
    double range[2][kMaxCluster * kMaxWarps];
    double warp[kMaxWarps];
    int test[kMaxK + 1];                // of a draft: 0 refused, 1 stands, 2 in doubt
    int first, last;
};

__device__ __forceinline__ double positive(double v) { return __double2hiint(v) < 0 ? 0.0 : v; } // (no NaN)

__device__ __forceinline__ uint64_t as_bits(float2 x)
{
    return (uint64_t)__float_as_uint(x.y) << 32 | __float_as_uint(x.x);
}
__device__ __forceinline__ float2 as_pair(uint64_t x)
{
    return make_float2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
}

// A stream's settings.
struct Stream {
    int drafts;
    float temperature;
    bool greedy;
    __device__ __forceinline__ Stream(const VerifyArgs &g, int64_t b)
    {
        drafts = g.n_draft ? min(max(g.n_draft[b], 0), g.K) : g.K;
        temperature = g.temperature ? g.temperature[b] : g.temperature_all;
        greedy = !(temperature > 0.0f);
        temperature = greedy ? 1.0f : fminf(temperature, 1.2676506e30f); // (2^100: differences of logits may be infinite)
    }
    __device__ __forceinline__ float per_t() const { return fminf(1.4426950408889634f / temperature, 3.4e38f); }
};

// Parts of a row, one to a lane (repeated every L lanes) -> the row's: maximum and sum, or the largest one's place.
template <int L> __device__ __forceinline__ uint64_t joined(uint64_t mine, bool greedy, float per_t)
{
    if (greedy) {
#pragma unroll
        for (int o = L / 2; o; o >>= 1) {
            const uint64_t y = __shfl_xor_sync(~0u, mine, o);
            mine = y > mine ? y : mine;
        }
        return mine;
    }
    const float2 x = as_pair(mine);
    float top = x.x;
#pragma unroll
    for (int o = L / 2; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    float sum = x.y * exp2_approx((x.x - top) * per_t);
#pragma unroll
    for (int o = L / 2; o; o >>= 1)
        sum += __shfl_xor_sync(~0u, sum, o);
    return as_bits(make_float2(top, sum));
}

template <typename T> __global__ void __launch_bounds__(kThreads) scan_kernel(const VerifyArgs g)
{
    constexpr int N = Vec<T>::N, kBatch = 8;
    __shared__ uint64_t parts[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    const int rows = g.draft ? 2 * g.K + 1 : g.K + 1;
    const uint32_t job = blockIdx.x / g.parts, part = blockIdx.x - job * g.parts;
    const int64_t b = job / rows;
    const int r = (int)(job - b * rows), place = r <= g.K ? r : r - (g.K + 1);
    const Stream st(g, b);
    if (r <= g.K ? place > st.drafts : place >= st.drafts)
        return;
    const T *row = (r <= g.K ? static_cast<const T *>(g.logits) + b * g.logits_batch + place * g.logits_row
                             : static_cast<const T *>(g.draft) + b * g.draft_batch + place * g.draft_row);
    const int begin = min(g.V, (int)part * g.part), n = min(g.part, g.V - begin);
    const T *p = row + begin;
    const int head = min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T)), nv = (n - head) / N;
    const uint4 *vec = reinterpret_cast<const uint4 *>(p + head);
    const float per_t = st.per_t();
    const bool greedy = st.greedy;
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
                        const uint64_t at = (uint64_t)order_key(x[k]) << 32 | (uint32_t)~(idx + k);
                        best = at > best ? at : best;
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
    for (int c0 = tid; c0 < nv; c0 += kThreads * kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            if (c0 + kThreads * e < nv)
                v[e] = __ldg(vec + c0 + kThreads * e);
#pragma unroll
        for (int e = 0; e < kBatch; ++e)
            if (c0 + kThreads * e < nv) {
                float x[N];
                Vec<T>::split(v[e], x);
                take(x, N, begin + head + (c0 + kThreads * e) * N);
            }
    }
    for (int i = tid; i < n - nv * N; i += kThreads) { // the codes before the first vector and behind the last one
        const int at = i < head ? i : i + nv * N;
        const float x = Vec<T>::one(p + at);
        take(&x, 1, begin + at);
    }
    const uint64_t x = joined<32>(greedy ? best : as_bits(make_float2(m, z)), greedy, per_t);
    if (lane == 0)
        parts[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const uint64_t y = joined<kWarps>(parts[lane % kWarps], greedy, per_t);
        if (lane == 0)
            g.stats[(b * (2 * g.K + 1) + r) * g.parts + part] = y;
    }
}

template <typename T>
__global__ void __launch_bounds__(kMaxThreads) verify_kernel(const VerifyArgs g, int C)
{
    __shared__ Shared sh;
    const int threads = blockDim.x, warps = threads / 32, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int64_t b = blockIdx.x / C;
    const int begin = min(g.V, (int)rank * g.slice), n = min(g.slice, g.V - begin);
    const T *logits = static_cast<const T *>(g.logits) + b * g.logits_batch;
    const T *draft = g.draft ? static_cast<const T *>(g.draft) + b * g.draft_batch : nullptr;
    const float *u = g.u + b * (g.K + 1);
    const int32_t *codes = g.codes + b * g.K;
    const Stream st(g, b);
    const int drafts = st.drafts;
    const float temperature = st.temperature;
    const bool greedy = st.greedy;
    if (tid < 64)
        sh.steps[tid >> 5][tid & 31] = exp2((double)(tid & 31) / (tid < 32 ? 32.0 : (double)kTable));
    __syncthreads();
    for (int i = tid; i < kTable; i += threads)
        sh.table[i] = sh.steps[0][i >> 5] * sh.steps[1][i & 31];
    auto number = [](float v) TOK_INLINE { return v >= 0.0f ? fminf(v, 0.99999994f) : 0.0f; }; // in [0, 1); NaN: 0
    const Weights weight(sh.table, temperature);
    // This warp's range [lo, hi) of the slice.
    const int per = ((n + warps - 1) / warps + 31) / 32 * 32;
    auto warp_sum = [&](double v) TOK_INLINE {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v += __shfl_xor_sync(~0u, v, o);
        return v;
    };
    constexpr int kRanges = kMaxCluster * kMaxWarps, kEach = kRanges / 32; // of all CTAs' warps: lane l has kEach in order
    float2 p_row{}, q_row{};
    // This thread's draft, while the scan runs.
    int drafted = -1;
    float logit_p = 0.0f, logit_q = 0.0f;
    double v = 0.0;
    if (tid < drafts) {
        drafted = codes[tid];
        v = number(u[tid]);
        if (drafted >= 0 && drafted < g.V) {
            logit_p = Vec<T>::one(logits + (int64_t)tid * g.logits_row + drafted);
            if (draft)
                logit_q = Vec<T>::one(draft + (int64_t)tid * g.draft_row + drafted);
        }
    }

    // ---- The rows' statistics, then all tests. ----
    asm volatile("griddepcontrol.wait;" ::: "memory"); // the grid before has written them
    for (int i = warp; i < drafts + 1 + (draft ? drafts : 0); i += warps) {
        const int r = i <= drafts ? i : g.K + 1 + (i - drafts - 1);
        const uint64_t none = greedy ? 0 : as_bits(make_float2(kLowest, 0.0f));
        const int at = lane % kMaxParts;
        const uint64_t x = joined<kMaxParts>(at < g.parts ? g.stats[(b * (2 * g.K + 1) + r) * g.parts + at] : none, greedy,
                                             st.per_t());
        if (lane == 0) // greedy: the index's bits, inverted, and whether there is one
            sh.all[r] = greedy ? make_float2(__uint_as_float((uint32_t)x), x ? 1.0f : 0.0f) : as_pair(x);
    }
    __syncthreads();
    auto rows_of = [&](int at) TOK_INLINE {
        p_row = sh.all[at];
        if (draft && at < drafts)
            q_row = sh.all[g.K + 1 + at];
    };
    // All passes over the codes in one loop, as it is the length of the code that counts with few streams: the sums
    // of p's and q's weights, for a test in doubt or for the draw; of max(p - q, 0); of p's alone, where nothing is
    // left of that.
    enum { kTests, kSums, kRest, kAlone } step = kTests;
    const T *p = nullptr, *q = nullptr;
    int place = 0, but = -1; // the place that the code is drawn at; the code that is left out
    bool refused = false, again = false;
    double zp = 0.0, zq = 0.0, rp = 1.0, rq = 0.0, total = 0.0;
    auto emit = [&](int code) TOK_INLINE { g.out[b * (g.K + 1) + place] = code; };
    for (int passes = 0;; ++passes) {
        if (step == kTests) {
            // v eq / zq < ep / zp: with the scan's sums at once, with exact ones one at a time.  (eq is 0 where the
            // draft's row has no code.)
            if (again ? tid == place : tid < drafts) {
                rows_of(tid);
                int stands = 0;
                if (drafted < 0 || drafted >= g.V)
                    stands = 0;
                else if (greedy)
                    stands = p_row.y != 0.0f && (int)~__float_as_uint(p_row.x) == drafted;
                else {
                    auto exact = [&](float top, float logit) TOK_INLINE {
                        const Weights::Row r = weight.row(top);
                        return exact_weight(r.top, r.least, r.only_top, logit, temperature);
                    };
                    const double ep = exact(p_row.x, logit_p);
                    const double eq = draft ? exact(q_row.x, logit_q) : 1.0;
                    const double veq = v * eq, left = veq * (again ? zp : (double)p_row.y);
                    const double right = ep * (!draft ? 1.0 : again ? zq : (double)q_row.y);
                    // (Sums of infinite logits are no numbers and in doubt, too.)
                    stands = veq == 0.0 || ep == 0.0                                ? (int)(ep > 0.0)
                             : again || fabs(left - right) > kDoubt * right ? (int)(left < right)
                                                                                    : 2;
                }
                sh.test[tid] = stands;
            }
            __syncthreads();
            while (place < drafts && sh.test[place] == 1)
                ++place;
            again = place < drafts && sh.test[place] == 2;
            rows_of(place);
            refused = place < drafts;
            p = logits + (int64_t)place * g.logits_row;
            q = refused && draft ? draft + (int64_t)place * g.draft_row : nullptr;
            if (!again) {
                step = kSums;
                if (rank == 0)
                    for (int i = tid; i <= g.K; i += threads)
                        if (i != place)
                            g.out[b * (g.K + 1) + i] = i < place ? codes[i] : -1;
                if (rank == 0 && tid == 0)
                    g.accepted[b] = place;
                if (greedy) {
                    if (rank == 0 && tid == 0)
                        emit(p_row.y != 0.0f ? (int)~__float_as_uint(p_row.x) : -1);
                    return; // (before the first pass: no CTA reads another's memory)
                }
                if (refused && !draft && codes[place] >= begin)
                    but = codes[place] - begin; // (in this CTA's slice, or of no other use)
            }
        }
        // A warp's range, kCodes of each lane at a time, the next ones' loads under way.
        const Weights::Row rowp = weight.row(p_row.x), rowq = weight.row(q_row.x);
        const int lo = min(n, warp * per), hi = min(n, lo + per);
        double sp = 0.0, sq = 0.0;
        float x[kCodes], y[kCodes];
        auto fetch = [&](int i0) TOK_INLINE {
#pragma unroll
            for (int e = 0; e < kCodes; ++e) {
                const int i = i0 + 32 * e;
                x[e] = i < hi && i != but ? Vec<T>::one(p + begin + i) : -INFINITY;
                y[e] = i < hi && q ? Vec<T>::one(q + begin + i) : -INFINITY;
            }
        };
        fetch(lo + lane);
#pragma unroll 1
        for (int i0 = lo + lane; i0 < hi + lane; i0 += 32 * kCodes) {
            float xs[kCodes], ys[kCodes];
#pragma unroll
            for (int e = 0; e < kCodes; ++e) {
                xs[e] = x[e];
                ys[e] = y[e];
            }
            fetch(i0 + 32 * kCodes);
            double wp[kCodes], wq[kCodes];
#pragma unroll
            for (int e = 0; e < kCodes; ++e) {
                wp[e] = weight(rowp, xs[e]);
                wq[e] = weight(rowq, ys[e]);
            }
            if (step == kRest) {
#pragma unroll
                for (int e = 0; e < kCodes; ++e)
                    sp += positive(wp[e] * rp - wq[e] * rq);
            } else {
#pragma unroll
                for (int e = 0; e < kCodes; ++e) {
                    sp += wp[e];
                    sq += wq[e];
                }
            }
        }
        // The sums of all ranges of all CTAs, in order.
        sp = warp_sum(sp);
        sq = warp_sum(sq);
        double (&sums)[2][kMaxWarps] = sh.sums[passes & 1]; // (those of the pass before may be read yet, no earlier ones)
        if (lane == 0) {
            sums[0][warp] = sp;
            sums[1][warp] = sq;
        }
        if (C > 1)
            cluster_sync();
        else
            __syncthreads();
        for (int i = tid; i < 2 * kRanges; i += threads) {
            const int which = i / kRanges, j = i - which * kRanges, c = j / warps;
            const double *mine = &sums[which][j - c * warps];
            sh.range[which][j] = c >= C ? 0.0 : C > 1 ? __longlong_as_double((long long)ld_cluster64(mine, c)) : *mine;
        }
        __syncthreads();
        zp = zq = 0.0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            zp += sh.range[0][lane * kEach + e];
            zq += sh.range[1][lane * kEach + e];
        }
        zp = warp_sum(zp);
        zq = warp_sum(zq);
        if (step == kTests) {
            zp *= weight.unit(rowp);
            zq *= weight.unit(rowq);
            continue;
        }
        total = zp;
        if (step == kSums && q && zp > 0.0 && zq > 0.0) {
            step = kRest;
            rp = 1.0 / zp;
            rq = 1.0 / zq;
            continue;
        }
        if (total > 0.0 || !refused || step == kAlone)
            break;
        step = kAlone; // nothing is left: from p itself
        q = nullptr;
        but = -1;
    }
    if (C > 1) // until then no CTA ends, as others may read its sums
        cluster_sync();
    if (total == 0.0) {
        if (rank == 0 && tid == 0)
            emit(-1);
        return;
    }

    // ---- The draw. ----
    double target = (double)number(u[g.K]) * total;
    // The range that the target lies in; the last with a weight where rounding leaves the target behind all.
    double mine = 0.0;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
        mine += sh.range[0][lane * kEach + e];
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
        const double r = sh.range[0][lane * kEach + e];
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
    if (range / warps != (int)rank)
        return;
    // The thread whose share of it the target lies in, then the code.
    const int lo = min(n, range % warps * per), hi = min(n, lo + per);
    const int each = (hi - lo + threads - 1) / threads, i0 = min(hi, lo + tid * each), i1 = min(hi, i0 + each);
    const Weights::Row rowp = weight.row(p_row.x), rowq = weight.row(q_row.x);
    if (tid == 0) {
        sh.first = 0x7FFFFFFF;
        sh.last = -1;
    }
    double before = 0.0; // of the codes before this thread's
    int code = -1;
    for (int look = 0; look < 2; ++look) {
        double upto = before;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            double w = weight(rowp, i == but ? -INFINITY : Vec<T>::one(p + begin + i));
            if (step == kRest)
                w = positive(w * rp - weight(rowq, Vec<T>::one(q + begin + i)) * rq);
            upto += w;
            if (look && w > 0.0) {
                code = begin + i;
                if (upto > target)
                    break;
            }
        }
        if (look)
            break;
        const double share = upto;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(~0u, upto, o);
            if (lane >= o)
                upto += y;
        }
        if (lane == 31)
            sh.warp[warp] = upto;
        __syncthreads();
        before = upto - share;
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
    }
    emit(code);
}

// Parts of a row in the scan: of 16,000 codes or more.
int parts_of(int64_t V) { return (int)std::min<int64_t>(kMaxParts, std::max<int64_t>(1, V / 16000)); }

template <typename T> tok_status launch(VerifyArgs g, int64_t B, cudaStream_t stream)
{
    constexpr int N = Vec<T>::N;
    auto slice_of = [&](int c) { return ((g.V + c - 1) / c + N - 1) / N * N; };
    g.parts = parts_of(g.V);
    g.part = slice_of(g.parts);
    const int64_t jobs = B * (g.draft ? 2 * g.K + 1 : g.K + 1) * g.parts;
    scan_kernel<T><<<(unsigned)jobs, kThreads, 0, stream>>>(g);
    const tok_status st = launch_status();
    if (st != TOK_OK)
        return st;
    // With few streams an SM each for up to 8 CTAs of all threads that it takes (4 streams: 22 us, with 256 threads
    // 39), else as many small CTAs as are resident at a time.
    const int64_t most = std::min<int64_t>(kMaxCluster, std::max<int64_t>(1, g.V / 2048));
    const bool few = B * most <= 148;
    const int C = (int)(few ? most : std::min(most, std::max<int64_t>(1, kCtas * 148 / B)));
    g.slice = slice_of(C);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.blockDim = dim3(few ? kMaxThreads : kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<T>, g, C);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }
    return launch_status();
}

bool verify_dims_ok(int64_t B, int64_t K, int64_t V)
{
    return B >= 0 && B <= ((int64_t)1 << 20) && K >= 0 && K <= kMaxK && V >= 1 && V <= kMaxV;
}

int64_t verify_workspace(int64_t B, int64_t K, int64_t V) { return B * (2 * K + 1) * parts_of(V) * 8; }

} // namespace
} // namespace tok

extern "C" int64_t tok_verify_codes_workspace_size(int64_t B, int64_t K, int64_t V)
{
    return tok::verify_dims_ok(B, K, V) ? tok::verify_workspace(B, K, V) : -1;
}

extern "C" tok_status tok_verify_codes(const void *logits, const void *draft_logits, tok_dtype dtype,
                                       const int32_t *codes, const float *u, const int32_t *n_draft,
                                       const float *temperature, float temperature_all, int32_t *out,
                                       int32_t *accepted, int64_t B, int64_t K, int64_t V, int64_t logits_batch,
                                       int64_t logits_row, int64_t draft_batch, int64_t draft_row, void *workspace,
                                       int64_t workspace_bytes, cudaStream_t stream)
{
    using namespace tok;
    if (dtype != TOK_F32 && dtype != TOK_BF16)
        return TOK_ERR_DTYPE;
    const int64_t size = dtype == TOK_F32 ? 4 : 2;
    constexpr int64_t kStride = (int64_t)1 << 40;
    if (!verify_dims_ok(B, K, V))
        return TOK_ERR_SHAPE;
    if (K == 0)
        draft_logits = nullptr, codes = nullptr; // there is nothing of them
    for (int64_t s : {B > 1 ? logits_batch : 0, K > 0 ? logits_row : 0, draft_logits && B > 1 ? draft_batch : 0,
                      draft_logits && K > 1 ? draft_row : 0})
        if (s < 0 || s >= kStride)
            return TOK_ERR_SHAPE;
    if (B == 0)
        return TOK_OK;
    const int64_t need = verify_workspace(B, K, V);
    if (workspace_bytes < need)
        return TOK_ERR_SHAPE;
    if (!logits || !u || !out || !accepted || !workspace || (K > 0 && !codes))
        return TOK_ERR_NULL;
    if (!aligned(logits, size) || !aligned(draft_logits, size) || !aligned(codes, 4) || !aligned(u, 4) ||
        !aligned(n_draft, 4) || !aligned(temperature, 4) || !aligned(out, 4) || !aligned(accepted, 4) ||
        !aligned(workspace, 16))
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
    const Range outs[] = {{out, 4 * B * (K + 1)}, {accepted, 4 * B}, {workspace, need}};
    for (const Range &o : outs)
        for (const Range &i : ins)
            if (i.p && overlaps(i.p, i.bytes, o.p, o.bytes))
                return TOK_ERR_ALIAS;
    if (overlaps(out, 4 * B * (K + 1), accepted, 4 * B) || overlaps(out, 4 * B * (K + 1), workspace, need) ||
        overlaps(accepted, 4 * B, workspace, need))
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
    g.stats = static_cast<uint64_t *>(workspace);
    return dtype == TOK_F32 ? launch<float>(g, B, stream) : launch<__nv_bfloat16>(g, B, stream);
}
