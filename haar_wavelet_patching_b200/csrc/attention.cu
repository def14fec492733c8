// Cross attention to an encoder's states of another length: o = softmax(scale q k^T) v
// over the first len[b] keys of each batch entry, query heads in groups that share a key
// head; its gradients; and the split form for few queries.
//
// Warp-level kernels: every product runs on m16n8k16 tiles whose fragments come straight
// from global memory as 16-byte loads (see attention.cuh), so there is no staging.
//
// attn_rows_kernel (forward): 16 query rows of one key head (queries x the heads of its
// group) per CTA; its 4 warps take 16 keys each in turn with a running maximum and sum of
// their own, joined through shared memory.  The keys are split over `splits` CTAs; with
// more than one, attn_join_kernel adds up their partial results in split order.
#include <algorithm>
#include <initializer_list>

#include "attention.cuh"

namespace tok {
namespace {

constexpr int kRows = 16; // query rows per CTA
constexpr int kFwdWarps = 4;
constexpr int kKeyStep = 16;

// Keys [begin, end) of split s: equal shares in whole rounds of the CTA's warps.
__device__ __forceinline__ void split_range(int len, int splits, int s, int &begin, int &end)
{
    constexpr int unit = kFwdWarps * kKeyStep;
    const int rounds = (len + unit - 1) / unit, per = (rounds + splits - 1) / splits;
    begin = min(len, s * per * unit);
    end = min(len, begin + per * unit);
}

// NP = ceil(D / 64).
template <int NP>
__global__ void __launch_bounds__(kFwdWarps * 32) attn_rows_kernel(const AttnArgs a)
{
    constexpr int NC = 2 * NP;
    __shared__ float sm[kFwdWarps][kRows], sl[kFwdWarps][kRows];
    __shared__ float so[kFwdWarps][kRows][NP * 64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int tiles = (a.Nq * a.G + kRows - 1) / kRows;
    const int split = blockIdx.x % a.splits, tile = (int)(blockIdx.x / a.splits) % tiles;
    const int bh = (int)(blockIdx.x / a.splits) / tiles, b = bh / a.Hkv, hk = bh - b * a.Hkv;
    const int rows = a.Nq * a.G, r0 = tile * kRows;
    int k0, k1;
    split_range(key_count(a, b), a.splits, split, k0, k1);

    uint4 qlo[NC], qhi[NC];
    {
        const int lo = r0 + g, hi = lo + 8;
        load_chan<NC>(qlo, a.q.row(b, lo / a.G, hk * a.G + lo % a.G), lo < rows, 8 * c, a.D);
        load_chan<NC>(qhi, a.q.row(b, hi / a.G, hk * a.G + hi % a.G), hi < rows, 8 * c, a.D);
    }
    float acc[NP][8][4] = {};
    float mlo = -INFINITY, mhi = -INFINITY, llo = 0.0f, lhi = 0.0f;
    for (int kk = k0 + warp * kKeyStep; kk < k1; kk += kFwdWarps * kKeyStep) {
        uint4 kf[2][NC];
        RowFrag vf[NP];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int key = kk + 8 * t + g;
            load_chan<NC>(kf[t], a.k.row(b, key, hk), key < k1, 8 * c, a.D);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = kk + 2 * c + (i & 1) + 8 * (i >> 1);
            const __nv_bfloat16 *row = a.v.row(b, key, hk);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                vf[p].r[i] = load16(row + 64 * p + 8 * g, key < k1 && 64 * p + 8 * g < a.D);
        }
        float s[2][4] = {};
        mma_chan<NC>(s[0], qlo, qhi, kf[0]);
        mma_chan<NC>(s[1], qlo, qhi, kf[1]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[t][e] = kk + 8 * t + 2 * c + (e & 1) < k1 ? s[t][e] * a.scale2 : -INFINITY;
        // key kk is one of this split's, so both maxima are those of at least one key
        const float nlo = fmaxf(mlo, quad_max(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]))));
        const float nhi = fmaxf(mhi, quad_max(fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))));
        if (__any_sync(~0u, nlo > mlo || nhi > mhi)) {
            const float flo = nlo == -INFINITY ? 1.0f : exp2_fast(mlo - nlo);
            const float fhi = nhi == -INFINITY ? 1.0f : exp2_fast(mhi - nhi);
            llo *= flo;
            lhi *= fhi;
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[p][j][0] *= flo;
                    acc[p][j][1] *= flo;
                    acc[p][j][2] *= fhi;
                    acc[p][j][3] *= fhi;
                }
            mlo = nlo;
            mhi = nhi;
        }
        const float zlo = mlo == -INFINITY ? 0.0f : mlo, zhi = mhi == -INFINITY ? 0.0f : mhi;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t][0] = exp2_fast(s[t][0] - zlo);
            s[t][1] = exp2_fast(s[t][1] - zlo);
            s[t][2] = exp2_fast(s[t][2] - zhi);
            s[t][3] = exp2_fast(s[t][3] - zhi);
            llo += s[t][0] + s[t][1];
            lhi += s[t][2] + s[t][3];
        }
        // The weights enter the second product as bf16 (its operands share one type).
        const uint32_t pa[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
        for (int p = 0; p < NP; ++p)
            mma_rows(acc[p], pa, vf[p]);
    }
    llo = quad_sum(llo);
    lhi = quad_sum(lhi);
    if (c == 0) {
        sm[warp][g] = mlo;
        sm[warp][g + 8] = mhi;
        sl[warp][g] = llo;
        sl[warp][g + 8] = lhi;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = 64 * p + 16 * c + j;
            so[warp][g][d] = acc[p][j][0];
            so[warp][g][d + 8] = acc[p][j][1];
            so[warp][g + 8][d] = acc[p][j][2];
            so[warp][g + 8][d + 8] = acc[p][j][3];
        }
    __syncthreads();
    // Join the warps: 8 threads per row, 8 channels at a time.
    const int row = threadIdx.x >> 3, r = r0 + row;
    if (r >= rows)
        return;
    float m = -INFINITY, l = 0.0f, f[kFwdWarps];
#pragma unroll
    for (int w = 0; w < kFwdWarps; ++w)
        m = fmaxf(m, sm[w][row]);
#pragma unroll
    for (int w = 0; w < kFwdWarps; ++w) {
        f[w] = sm[w][row] == -INFINITY ? 0.0f : exp2_fast(sm[w][row] - m);
        l += f[w] * sl[w][row];
    }
    const int iq = r / a.G, h = hk * a.G + r % a.G;
    const int64_t stat = ((int64_t)b * a.Hq + h) * a.Nq + iq;
    const int64_t nstat = (int64_t)a.B * a.Hq * a.Nq;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    for (int d = 8 * (threadIdx.x & 7); d < a.D; d += 64) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = 0.0f;
#pragma unroll
            for (int w = 0; w < kFwdWarps; ++w)
                v[j] += f[w] * so[w][row][d + j];
        }
        if (a.splits == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] *= inv;
            Row<__nv_bfloat16, 8, true>::store(a.o.row(b, iq, h) + d, v);
        } else
            Row<float, 8, true>::store(a.part + (split * nstat + stat) * a.D + d, v);
    }
    if ((threadIdx.x & 7) == 0) {
        if (a.splits == 1) {
            if (a.lse)
                a.lse[stat] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        } else {
            float *ml = a.part + a.splits * nstat * a.D + 2 * (split * nstat + stat);
            ml[0] = m;
            ml[1] = l;
        }
    }
}

// One warp per query row and head: the splits' partial results in split order.
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a)
{
    const int64_t nstat = (int64_t)a.B * a.Hq * a.Nq;
    const int64_t stat = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (stat >= nstat)
        return;
    const float *ml = a.part + a.splits * nstat * a.D;
    float m = -INFINITY, l = 0.0f;
    for (int s = 0; s < a.splits; ++s)
        m = fmaxf(m, ml[2 * (s * nstat + stat)]);
    float v[4] = {};
    const int d = 4 * lane;
    for (int s = 0; s < a.splits; ++s) {
        const float ms = ml[2 * (s * nstat + stat)];
        if (ms == -INFINITY)
            continue;
        const float f = exp2_fast(ms - m);
        l += f * ml[2 * (s * nstat + stat) + 1];
        if (d < a.D) {
            float x[4];
            Row<float, 4, true>::load(a.part + (s * nstat + stat) * a.D + d, x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] += f * x[j];
        }
    }
    const int iq = (int)(stat % a.Nq), bh = (int)(stat / a.Nq), b = bh / a.Hq, h = bh - b * a.Hq;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    if (d < a.D) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] *= inv;
        Row<__nv_bfloat16, 4, true>::store(a.o.row(b, iq, h) + d, v);
    }
    if (lane == 0 && a.lse)
        a.lse[stat] = l > 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// delta = rowsum(go * o) of every query row: 8 lanes per row.
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnArgs a)
{
    const int64_t stat = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    const int c = threadIdx.x & 7;
    const bool live = stat < (int64_t)a.B * a.Hq * a.Nq;
    float s = 0.0f;
    if (live) { // heads of a token lie next to each other
        const int h = (int)(stat % a.Hq), iq = (int)(stat / a.Hq % a.Nq), b = (int)(stat / a.Hq / a.Nq);
        for (int d = 8 * c; d < a.D; d += 64) {
            float x[8], y[8];
            Row<__nv_bfloat16, 8, true>::load(a.go.row(b, iq, h) + d, x);
            Row<__nv_bfloat16, 8, true>::load(a.o.row(b, iq, h) + d, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s = fmaf(x[j], y[j], s);
        }
        s += __shfl_xor_sync(__activemask(), s, 1);
        s += __shfl_xor_sync(__activemask(), s, 2);
        s += __shfl_xor_sync(__activemask(), s, 4);
        if (c == 0)
            a.delta[((int64_t)b * a.Hq + h) * a.Nq + iq] = s;
    }
}

// dq = scale * ds k with ds = p (go v^T - delta): one warp per 16 query rows, over all keys.
template <int NP> __global__ void __launch_bounds__(128) attn_dq_kernel(const AttnArgs a)
{
    constexpr int NC = 2 * NP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int rows = a.Nq * a.G, tiles = (rows + 4 * kRows - 1) / (4 * kRows);
    const int tile = (int)blockIdx.x % tiles, bh = (int)blockIdx.x / tiles, b = bh / a.Hkv, hk = bh - b * a.Hkv;
    const int lo = (tile * 4 + warp) * kRows + g, hi = lo + 8, len = key_count(a, b);
    const int iqlo = lo / a.G, hlo = hk * a.G + lo % a.G, iqhi = hi / a.G, hhi = hk * a.G + hi % a.G;
    uint4 qlo[NC], qhi[NC], glo[NC], ghi[NC];
    load_chan<NC>(qlo, a.q.row(b, iqlo, hlo), lo < rows, 8 * c, a.D);
    load_chan<NC>(qhi, a.q.row(b, iqhi, hhi), hi < rows, 8 * c, a.D);
    load_chan<NC>(glo, a.go.row(b, iqlo, hlo), lo < rows, 8 * c, a.D);
    load_chan<NC>(ghi, a.go.row(b, iqhi, hhi), hi < rows, 8 * c, a.D);
    const int64_t slo = ((int64_t)b * a.Hq + hlo) * a.Nq + iqlo, shi = ((int64_t)b * a.Hq + hhi) * a.Nq + iqhi;
    const float l2lo = lo < rows ? a.lse_in[slo] * 1.4426950408889634f : 0.0f;
    const float l2hi = hi < rows ? a.lse_in[shi] * 1.4426950408889634f : 0.0f;
    const float dlo = lo < rows ? a.delta[slo] : 0.0f, dhi = hi < rows ? a.delta[shi] : 0.0f;
    float acc[NP][8][4] = {};
    for (int kk = 0; kk < len; kk += kKeyStep) {
        uint4 kf[2][NC], vf[2][NC];
        RowFrag kr[NP];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int key = kk + 8 * t + g;
            load_chan<NC>(kf[t], a.k.row(b, key, hk), key < len, 8 * c, a.D);
            load_chan<NC>(vf[t], a.v.row(b, key, hk), key < len, 8 * c, a.D);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = kk + 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                kr[p].r[i] = load16(a.k.row(b, key, hk) + 64 * p + 8 * g, key < len && 64 * p + 8 * g < a.D);
        }
        float s[2][4] = {}, dp[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            mma_chan<NC>(s[t], qlo, qhi, kf[t]);
            mma_chan<NC>(dp[t], glo, ghi, vf[t]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = kk + 8 * t + 2 * c + (e & 1) < len;
                const float p = exp2_fast(fmaf(s[t][e], a.scale2, e < 2 ? -l2lo : -l2hi));
                s[t][e] = in ? p * (dp[t][e] - (e < 2 ? dlo : dhi)) : 0.0f;
            }
        }
        const uint32_t ds[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
#pragma unroll
        for (int p = 0; p < NP; ++p)
            mma_rows(acc[p], ds, kr[p]);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = e < 2 ? lo : hi, d = 64 * p + 16 * c + 8 * (e & 1);
            if (r < rows && d < a.D) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = acc[p][j][e] * a.scale;
                Row<__nv_bfloat16, 8, true>::store(
                    (e < 2 ? a.dq.row(b, iqlo, hlo) : a.dq.row(b, iqhi, hhi)) + d, v);
            }
        }
}

// dv = p^T go and dk = scale * ds^T q: one warp per 16 keys of a key head, over the queries
// of all heads of its group in order.
template <int NP> __global__ void __launch_bounds__(128) attn_dkv_kernel(const AttnArgs a)
{
    constexpr int NC = 2 * NP;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int tiles = (a.Nk + 4 * kKeyStep - 1) / (4 * kKeyStep);
    const int tile = (int)blockIdx.x % tiles, bh = (int)blockIdx.x / tiles, b = bh / a.Hkv, hk = bh - b * a.Hkv;
    const int len = key_count(a, b), lo = (tile * 4 + warp) * kKeyStep + g, hi = lo + 8;
    uint4 klo[NC], khi[NC], vlo[NC], vhi[NC];
    load_chan<NC>(klo, a.k.row(b, lo, hk), lo < len, 8 * c, a.D);
    load_chan<NC>(khi, a.k.row(b, hi, hk), hi < len, 8 * c, a.D);
    load_chan<NC>(vlo, a.v.row(b, lo, hk), lo < len, 8 * c, a.D);
    load_chan<NC>(vhi, a.v.row(b, hi, hk), hi < len, 8 * c, a.D);
    float dk[NP][8][4] = {}, dv[NP][8][4] = {};
    const bool any = (tile * 4 + warp) * kKeyStep < len;
    for (int h = hk * a.G; any && h < (hk + 1) * a.G; ++h) {
        const int64_t stat = ((int64_t)b * a.Hq + h) * a.Nq;
        for (int qq = 0; qq < a.Nq; qq += 16) {
            uint4 qf[2][NC], gf[2][NC];
            float st[2][4] = {}, dp[2][4] = {};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int iq = qq + 8 * t + g;
                load_chan<NC>(qf[t], a.q.row(b, iq, h), iq < a.Nq, 8 * c, a.D);
                load_chan<NC>(gf[t], a.go.row(b, iq, h), iq < a.Nq, 8 * c, a.D);
                mma_chan<NC>(st[t], klo, khi, qf[t]);
                mma_chan<NC>(dp[t], vlo, vhi, gf[t]);
            }
            uint32_t pa[4], ds[4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float p[4], d[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int iq = qq + 8 * t + 2 * c + (e & 1);
                    const bool in = iq < a.Nq && (e < 2 ? lo : hi) < len;
                    const float l2 = iq < a.Nq ? a.lse_in[stat + iq] * 1.4426950408889634f : 0.0f;
                    const float de = iq < a.Nq ? a.delta[stat + iq] : 0.0f;
                    p[e] = in ? exp2_fast(fmaf(st[t][e], a.scale2, -l2)) : 0.0f;
                    d[e] = in ? p[e] * (dp[t][e] - de) : 0.0f;
                }
                pa[2 * t] = pack_bf16x2(p[0], p[1]);
                pa[2 * t + 1] = pack_bf16x2(p[2], p[3]);
                ds[2 * t] = pack_bf16x2(d[0], d[1]);
                ds[2 * t + 1] = pack_bf16x2(d[2], d[3]);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                RowFrag gr, qr;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int iq = qq + 2 * c + (i & 1) + 8 * (i >> 1);
                    const bool ok = iq < a.Nq && 64 * p + 8 * g < a.D;
                    gr.r[i] = load16(a.go.row(b, iq, h) + 64 * p + 8 * g, ok);
                    qr.r[i] = load16(a.q.row(b, iq, h) + 64 * p + 8 * g, ok);
                }
                mma_rows(dv[p], pa, gr);
                mma_rows(dk[p], ds, qr);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = e < 2 ? lo : hi, d = 64 * p + 16 * c + 8 * (e & 1);
            if (key < a.Nk && d < a.D) { // keys past the length: zeros
                float x[8], y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = dk[p][j][e] * a.scale;
                    y[j] = dv[p][j][e];
                }
                Row<__nv_bfloat16, 8, true>::store(a.dk.row(b, key, hk) + d, x);
                Row<__nv_bfloat16, 8, true>::store(a.dv.row(b, key, hk) + d, y);
            }
        }
}

// ---------------------------------------------------------------------------
// Host: argument rules.
// ---------------------------------------------------------------------------
constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;

struct Dims {
    int64_t B, Nq, Nk, Hq, Hkv, D;
    bool ok() const
    {
        int64_t p;
        return B >= 0 && Nq >= 0 && Nk >= 0 && Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0 && D >= 8 && D <= 128 &&
               D % 8 == 0 && Nq <= kIntMax - 1024 && Nk <= kIntMax - 1024 && Hq <= 65535 && B <= 65535 &&
               prod_ok({B, Hq, Nq}, &p) && p <= kIntMax / 2 && prod_ok({B, Hkv, Nk}, &p) && p <= kIntMax / 2 &&
               prod_ok({Hq, Nq}, &p) && p <= kIntMax / 2;
    }
};

struct Axis {
    int64_t n, s;
};

// No element of the strided dims (dense block of D) is met twice: each stride leaves room
// for everything of smaller stride.
bool nested(std::initializer_list<Axis> dims, int64_t D)
{
    Axis a[4];
    int n = 0;
    for (const Axis &x : dims)
        if (x.n > 1)
            a[n++] = x;
    std::sort(a, a + n, [](const Axis &x, const Axis &y) { return x.s < y.s; });
    int64_t span = D;
    for (int i = 0; i < n; ++i) {
        if (a[i].s < span)
            return false;
        span += (a[i].n - 1) * a[i].s;
    }
    return true;
}

struct View {
    const tok_heads *t;
    int64_t B, N, H, D;
    int64_t span() const { return (B - 1) * t->batch + (N - 1) * t->token + (H - 1) * t->head + D; }
    bool strides_ok() const
    {
        constexpr int64_t kMax = (int64_t)1 << 38; // elements: byte strides and spans stay far inside 64 bits
        for (const Axis &x : {Axis{B, t->batch}, Axis{N, t->token}, Axis{H, t->head}})
            if (x.n > 1 && (x.s < 0 || x.s >= kMax))
                return false;
        return true;
    }
    bool distinct() const { return nested({{B, t->batch}, {N, t->token}, {H, t->head}}, D); }
    bool aligned16() const
    {
        for (const Axis &x : {Axis{B, t->batch}, Axis{N, t->token}, Axis{H, t->head}})
            if (x.n > 1 && x.s % 8)
                return false;
        return aligned(t->ptr, 16);
    }
};

// Whether two views may share an element: their ranges meet, and they are not slices that
// interleave (equal strides, and the distance between them fits into the gaps).
bool meet(const View &a, const View &b)
{
    if (!overlaps(a.t->ptr, a.span() * 2, b.t->ptr, b.span() * 2))
        return false;
    const int64_t off = ((const char *)b.t->ptr - (const char *)a.t->ptr) / 2;
    auto same = [](int64_t na, int64_t sa, int64_t nb, int64_t sb) { return na <= 1 || nb <= 1 || sa == sb; };
    if (!same(a.B, a.t->batch, b.B, b.t->batch) || !same(a.N, a.t->token, b.N, b.t->token) ||
        !same(a.H, a.t->head, b.H, b.t->head))
        return true;
    auto ax = [](int64_t na, int64_t sa, int64_t nb, int64_t sb) { return Axis{std::max(na, nb), na > 1 ? sa : sb}; };
    return !nested({ax(a.B, a.t->batch, b.B, b.t->batch), ax(a.N, a.t->token, b.N, b.t->token),
                    ax(a.H, a.t->head, b.H, b.t->head), Axis{2, off < 0 ? -off : off}},
                   a.D);
}

bool meets(const View &a, const void *p, int64_t bytes) { return p && overlaps(a.t->ptr, a.span() * 2, p, bytes); }

HeadsView view(const tok_heads *t)
{
    return HeadsView{static_cast<__nv_bfloat16 *>(t->ptr), t->batch, t->token, t->head};
}

// Query rows per key head from which the tensor-core kernel takes a call.
constexpr int64_t kTcRows = 64;

bool wants_tc(const Dims &d) { return d.Nq * (d.Hq / d.Hkv) > kTcRows && d.Nk > 0; }

// CTAs that the keys of one row tile are split over.
int64_t fwd_splits(const Dims &d)
{
    const int64_t G = d.Hq / d.Hkv;
    if (wants_tc(d)) { // one CTA per SM, each with at least four key tiles
        const int64_t gp = attn_tc_group((int)G), items = d.B * (d.Hq / gp) * ((d.Nq * gp + 255) / 256);
        if (items == 0)
            return 1;
        return std::max<int64_t>(1, std::min(148 / items, d.Nk / 512));
    }
    // Four CTAs per SM, each with at least four rounds of its warps.
    const int64_t tiles = (d.Nq * G + kRows - 1) / kRows, units = d.B * d.Hkv * tiles;
    if (units == 0)
        return 1;
    const int64_t want = (148 * 4 + units - 1) / units, most = d.Nk / (4 * kFwdWarps * kKeyStep);
    return std::max<int64_t>(1, std::min(std::min(want, most), (int64_t)64));
}

} // namespace
} // namespace tok

extern "C" int64_t tok_cross_attention_workspace_size(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv,
                                                      int64_t D)
{
    const tok::Dims d{B, Nq, Nk, Hq, Hkv, D};
    if (!d.ok())
        return -1;
    const int64_t s = tok::fwd_splits(d);
    return s > 1 ? s * B * Hq * Nq * (D + 2) * 4 : 0;
}

extern "C" int64_t tok_cross_attention_backward_workspace_size(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq,
                                                               int64_t Hkv, int64_t D)
{
    const tok::Dims d{B, Nq, Nk, Hq, Hkv, D};
    return d.ok() ? B * Hq * Nq * 4 : -1;
}

extern "C" tok_status tok_cross_attention(const tok_heads *q, const tok_heads *k, const tok_heads *v,
                                          const tok_heads *o, float *lse, const int32_t *k_lens, int64_t B,
                                          int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D, float scale,
                                          void *workspace, int64_t workspace_bytes, cudaStream_t stream)
{
    using namespace tok;
    const Dims dim{B, Nq, Nk, Hq, Hkv, D};
    if (!dim.ok())
        return TOK_ERR_SHAPE;
    if (B == 0 || Nq == 0)
        return TOK_OK;
    if (!q || !k || !v || !o || !q->ptr || !o->ptr || (Nk > 0 && (!k->ptr || !v->ptr)))
        return TOK_ERR_NULL;
    const int64_t splits = fwd_splits(dim), need = tok_cross_attention_workspace_size(B, Nq, Nk, Hq, Hkv, D);
    const View vq{q, B, Nq, Hq, D}, vk{k, B, Nk, Hkv, D}, vv{v, B, Nk, Hkv, D}, vo{o, B, Nq, Hq, D};
    for (const View &x : {vq, vk, vv, vo})
        if (!x.strides_ok())
            return TOK_ERR_SHAPE;
    if (!vo.distinct() || workspace_bytes < need)
        return TOK_ERR_SHAPE;
    if (need > 0 && !workspace)
        return TOK_ERR_NULL;
    for (const View &x : {vq, vk, vv, vo})
        if (!x.aligned16())
            return TOK_ERR_ALIGN;
    if (!aligned(lse, 4) || !aligned(k_lens, 4) || (need > 0 && !aligned(workspace, 16)))
        return TOK_ERR_ALIGN;
    const int64_t stats = B * Hq * Nq * 4;
    const void *ws = need > 0 ? workspace : nullptr;
    if (meet(vo, vq) || (Nk > 0 && (meet(vo, vk) || meet(vo, vv))) || meets(vo, lse, stats) ||
        meets(vo, k_lens, 4 * B) || meets(vo, ws, need) || meets(vq, lse, stats) || meets(vq, ws, need) ||
        (Nk > 0 && (meets(vk, lse, stats) || meets(vv, lse, stats) || meets(vk, ws, need) || meets(vv, ws, need))) ||
        (lse && ((ws && overlaps(lse, stats, ws, need)) || (k_lens && overlaps(lse, stats, k_lens, 4 * B)))) ||
        (ws && k_lens && overlaps(ws, need, k_lens, 4 * B)))
        return TOK_ERR_ALIAS;

    AttnArgs a{};
    a.q = view(q);
    a.k = view(k);
    a.v = view(v);
    a.o = view(o);
    a.lse = lse;
    a.lens = k_lens;
    a.part = static_cast<float *>(workspace);
    a.B = (int)B;
    a.Nq = (int)Nq;
    a.Nk = (int)Nk;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.D = (int)D;
    a.splits = (int)splits;
    a.scale = scale;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    const int64_t blocks = B * Hkv * ((Nq * a.G + kRows - 1) / kRows) * splits;
    tok_status st;
    if (wants_tc(dim) && !attn_tc_broadcast_tokens(a)) {
        st = attn_tc_forward(a, stream);
    } else if (D <= 64) {
        attn_rows_kernel<1><<<(unsigned)blocks, kFwdWarps * 32, 0, stream>>>(a);
        st = launch_status();
    } else {
        attn_rows_kernel<2><<<(unsigned)blocks, kFwdWarps * 32, 0, stream>>>(a);
        st = launch_status();
    }
    if (st == TOK_OK && splits > 1) {
        attn_join_kernel<<<(unsigned)((B * Hq * Nq + 3) / 4), 128, 0, stream>>>(a);
        st = launch_status();
    }
    return st;
}

extern "C" tok_status tok_cross_attention_backward(const tok_heads *q, const tok_heads *k, const tok_heads *v,
                                                   const tok_heads *o, const float *lse, const tok_heads *grad_o,
                                                   const int32_t *k_lens, const tok_heads *grad_q,
                                                   const tok_heads *grad_k, const tok_heads *grad_v, int64_t B,
                                                   int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D,
                                                   float scale, void *workspace, int64_t workspace_bytes,
                                                   cudaStream_t stream)
{
    using namespace tok;
    const Dims dim{B, Nq, Nk, Hq, Hkv, D};
    if (!dim.ok())
        return TOK_ERR_SHAPE;
    if (B == 0 || (Nq == 0 && Nk == 0))
        return TOK_OK;
    for (const tok_heads *t : {q, k, v, o, grad_o, grad_q, grad_k, grad_v})
        if (!t)
            return TOK_ERR_NULL;
    if ((Nq > 0 && (!q->ptr || !o->ptr || !lse || !grad_o->ptr || !grad_q->ptr)) ||
        (Nk > 0 && (!k->ptr || !v->ptr || !grad_k->ptr || !grad_v->ptr)))
        return TOK_ERR_NULL;
    const int64_t need = tok_cross_attention_backward_workspace_size(B, Nq, Nk, Hq, Hkv, D);
    const View ins[] = {{q, B, Nq, Hq, D}, {o, B, Nq, Hq, D}, {grad_o, B, Nq, Hq, D}, {k, B, Nk, Hkv, D}, {v, B, Nk, Hkv, D}};
    const View outs[] = {{grad_q, B, Nq, Hq, D}, {grad_k, B, Nk, Hkv, D}, {grad_v, B, Nk, Hkv, D}};
    for (const View &x : ins)
        if (!x.strides_ok())
            return TOK_ERR_SHAPE;
    for (const View &x : outs)
        if (!x.strides_ok() || !x.distinct())
            return TOK_ERR_SHAPE;
    if (workspace_bytes < need)
        return TOK_ERR_SHAPE;
    if (need > 0 && !workspace)
        return TOK_ERR_NULL;
    for (const View &x : ins)
        if (!x.aligned16())
            return TOK_ERR_ALIGN;
    for (const View &x : outs)
        if (!x.aligned16())
            return TOK_ERR_ALIGN;
    if (!aligned(lse, 4) || !aligned(k_lens, 4) || !aligned(workspace, 16))
        return TOK_ERR_ALIGN;
    const int64_t stats = B * Hq * Nq * 4;
    for (int i = 0; i < 3; ++i) {
        if (outs[i].N == 0)
            continue;
        for (const View &x : ins)
            if (x.N > 0 && meet(outs[i], x))
                return TOK_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (outs[j].N > 0 && meet(outs[i], outs[j]))
                return TOK_ERR_ALIAS;
        if ((Nq > 0 && meets(outs[i], lse, stats)) || meets(outs[i], k_lens, 4 * B) ||
            (need > 0 && meets(outs[i], workspace, need)))
            return TOK_ERR_ALIAS;
    }
    if (need > 0) {
        for (const View &x : ins)
            if (x.N > 0 && meets(x, workspace, need))
                return TOK_ERR_ALIAS;
        if (overlaps(lse, stats, workspace, need) || (k_lens && overlaps(k_lens, 4 * B, workspace, need)))
            return TOK_ERR_ALIAS;
    }

    AttnArgs a{};
    a.q = view(q);
    a.k = view(k);
    a.v = view(v);
    a.o = view(o);
    a.go = view(grad_o);
    a.dq = view(grad_q);
    a.dk = view(grad_k);
    a.dv = view(grad_v);
    a.lse_in = lse;
    a.delta = static_cast<float *>(workspace);
    a.lens = k_lens;
    a.B = (int)B;
    a.Nq = (int)Nq;
    a.Nk = (int)Nk;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.D = (int)D;
    a.splits = 1;
    a.scale = scale;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    tok_status st = TOK_OK;
    if (Nq > 0) {
        attn_delta_kernel<<<(unsigned)((B * Hq * Nq + 31) / 32), 256, 0, stream>>>(a);
        st = launch_status();
        const unsigned blocks = (unsigned)(B * Hkv * ((Nq * a.G + 4 * kRows - 1) / (4 * kRows)));
        if (st == TOK_OK) {
            if (D <= 64)
                attn_dq_kernel<1><<<blocks, 128, 0, stream>>>(a);
            else
                attn_dq_kernel<2><<<blocks, 128, 0, stream>>>(a);
            st = launch_status();
        }
    }
    if (st == TOK_OK && Nk > 0) {
        const unsigned blocks = (unsigned)(B * Hkv * ((Nk + 4 * kKeyStep - 1) / (4 * kKeyStep)));
        if (D <= 64)
            attn_dkv_kernel<1><<<blocks, 128, 0, stream>>>(a);
        else
            attn_dkv_kernel<2><<<blocks, 128, 0, stream>>>(a);
        st = launch_status();
    }
    return st;
}
