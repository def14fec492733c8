// Gradients of cross attention on the 5th-generation tensor cores.
//
//   p = 2^(scale2 q k^T - lse2),  dp = go v^T,  ds = p (dp - delta),  delta = rowsum(go o)
//   dv = p^T go,  dk = scale ds^T q,  dq = scale ds k
//
// Two passes that each recompute p and dp, 7 products for the 5 of the formulas: a single
// pass would have to add up dq (or dk and dv) across CTAs, with atomics (whose order would
// show in the result) or with a partial result per key tile (Nk / 128 times dq in fp32
// through HBM).
//
// Query rows go in tiles of 128 as in the forward (G heads x 128 / G tokens of one group
// where G is a power of two, else 128 tokens of one head).  attn_stats_kernel lays out lse2 and
// delta in that order, padded to whole tiles (+inf and 0: p = 0 there).
//
// attn_dkv_kernel: one CTA per tile of 128 keys and share of the query tiles; s^T = k q^T and
//   dp^T = v go^T have a key per tensor-memory lane, so p^T and ds^T are the A operands of
//   dv += p^T go and dk += ds^T q as they stand.  q and go are read by two products each:
//   [row][channel] tiles serve as K-major and as MN-major operand.  Once dp^T is in registers, p^T and
//   ds^T both go over its columns, so that s(i+1) can follow as soon as s(i) has been read; the powers
//   of i+1 run under dv(i), dk(i) and dp(i+1).  With shares, partial sums go to fp32 and
//   attn_dkv_sum_kernel adds them in order.
// attn_dq_kernel: one CTA per SM walks the query tiles (and, with few of them, shares of the keys, added up
//   by attn_dq_sum_kernel); per key tile s, dp and dq += ds k,
//   s double-buffered so that s(i+2), dp(i+1) and dq(i) run under the arithmetic of i+1.
// delta comes from the o that is given, rounded to bf16, an error of up to 2^-8 |go| |o| that averages out over many keys but
// not over few: where a batch entry has at most 128 keys, attn_dq_kernel (which runs first) has
// all of a row's p and dp at hand and takes delta = sum p dp from them.
// In both, two warpgroups take half of a tile's columns each.
// Measured, 16 heads of 128, 2 x 3520 queries x 3520 keys: statistics 10 us, dq 291 + 5, dkv 385 + 6 (the
// second figures are the sums of the last rounds' shares): 690 us, 1030 TFLOP/s for the 7 products.
// 4 x 7040 x 512 ragged keys, 16 heads of 64 on 4: 27, 116, 134 + 6 us.  Both are bound by the chain
// of a tile (products -> arithmetic -> products) and, run for long, by the power limit.
#include <algorithm>

#include "attention.cuh"

namespace tok {

static __device__ unsigned int g_attn_bwd_timeouts = 0;

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 384; // warps 0-7 arithmetic, 8 MMA, 9 copies; 10 and 11 make the register split whole
constexpr int kMathRegs = 208, kOtherRegs = 88;
constexpr uint32_t SUB = kTile * 128; // bytes of 128 rows x 64 channels
constexpr float kLog2e = 1.4426950408889634f;

template <int DP> constexpr uint32_t tile_bytes() { return kTile * DP * 2; }

struct BwdArgs {
    AttnArgs a;
    const float *lse2; // [B][hsets][rows]
    float *delta;      // likewise
    float *part;               // [shares][2][tail][128][D]
    int gp, lgp;               // heads per tile: a power of two
    int hsets, rows;           // Hq / gp, padded query rows of a head set
    int qtiles;                // rows / 128
    FastDiv qtiles_div, hsets_div;
    int wide, dq_wide;         // rows of dk and dv, of dq start on 32 bytes
    int ktiles;                // ceil(Nk / 128)
    int hs_kv;                 // head sets per key head
    int whole, tail;           // dkv: key tiles that one CTA takes, then ones that several share
    int shares, per;           // of these: shares, query tiles (over hs_kv sets) of a share
    int dq_whole, dq_tail;     // dq: likewise query tiles,
    int dq_shares, dq_per;     // and key tiles of a share
    int dq_items;              // dq_whole + dq_tail * dq_shares
    float *dq_part;            // [dq_shares][dq_tail][128][D]
    int qb, gb, kb, kh, vb, vh;
};

// lse2 and delta of every query row, in tile order: a block per tile of 128, 8 lanes per row, four rows in
// flight per lane.
constexpr int kStatRows = kTile / 32;
template <int DP> __global__ void __launch_bounds__(256) attn_stats_kernel(const BwdArgs t, float *lse2, float *delta)
{
    const AttnArgs &a = t.a;
    const int c = threadIdx.x & 7;
    const int set = t.qtiles_div.div(blockIdx.x), tile = (int)blockIdx.x - set * t.qtiles;
    const int b = t.hsets_div.div(set), h0 = (set - b * t.hsets) * t.gp, lgp = t.lgp;
    const int r0 = tile * kTile + (int)(threadIdx.x >> 3);
    const int64_t at0 = (int64_t)blockIdx.x * kTile + (threadIdx.x >> 3);
    constexpr int NSUB = DP / 64;
    uint4 x[kStatRows][NSUB], y[kStatRows][NSUB];
    float l[kStatRows];
#pragma unroll
    for (int k = 0; k < kStatRows; ++k) {
        const int r = r0 + 32 * k, h = h0 + (r & (t.gp - 1)), iq = r >> lgp;
        const bool live = iq < a.Nq;
#pragma unroll
        for (int e = 0; e < NSUB; ++e) {
            const int d = 8 * c + 64 * e;
            x[k][e] = load16(a.go.row(b, iq, h) + d, live && d < a.D);
            y[k][e] = load16(a.o.row(b, iq, h) + d, live && d < a.D);
        }
        l[k] = live && c == 0 ? a.lse_in[((int64_t)b * a.Hq + h) * a.Nq + iq] * kLog2e : INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kStatRows; ++k) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < NSUB; ++e)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                s = fmaf(bf16_lo(word(x[k][e], w)), bf16_lo(word(y[k][e], w)), s);
                s = fmaf(bf16_hi(word(x[k][e], w)), bf16_hi(word(y[k][e], w)), s);
            }
        s += __shfl_xor_sync(~0u, s, 1);
        s += __shfl_xor_sync(~0u, s, 2);
        s += __shfl_xor_sync(~0u, s, 4);
        const int64_t at = at0 + 32 * k;
        if (c == 0) {
            lse2[at] = l[k] == -INFINITY ? INFINITY : l[k]; // (a row without a key)
            delta[at] = s;
        }
    }
}

template <int DP> struct DkvSmem {
    static constexpr int NQ = DP == 128 ? 2 : 4, NG = NQ; // stages of q and go
    static constexpr uint32_t TB = tile_bytes<DP>();
    static constexpr uint32_t k = 0, v = TB, q = 2 * TB, g = q + NQ * TB, st = g + NG * TB; // stats: NQ x 1 KB
    static constexpr size_t bytes = st + NQ * 1024 + 1024;
};

struct Words8 {
    uint32_t w[8];
};
__device__ __forceinline__ Words8 packed(const uint32_t *x) // 16 fp32 -> bf16
{
    Words8 r;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        r.w[k] = pack_bf16x2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
    return r;
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const Words8 &v, int left, bool wide) { tok::store16(p, v.w, left, wide); }
__device__ __forceinline__ void store16(float *p, const uint32_t *x, int left)
{
    const float *v = reinterpret_cast<const float *>(x);
    if (left > 0)
        Row<float, 8, true>::store(p, v);
    if (left >= 16)
        Row<float, 8, true>::store(p + 8, v + 8);
}

// [row][channel] tile as K-major operand, byte offset of K step k (16 channels).
__device__ __forceinline__ constexpr uint32_t kmajor_step(int k) { return (k / 4) * SUB + (k % 4) * 32; }

// Half a tile's columns of one lane: 64 columns of tensor memory.
__device__ __forceinline__ void load_half(uint32_t col, float (&x)[64])
{
    tmem_ld64(col, reinterpret_cast<uint32_t(&)[64]>(x));
    tmem_wait_ld();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_dkv_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap gmap,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const BwdArgs t)
{
    using L = DkvSmem<DP>;
    constexpr int NQ = L::NQ, NG = L::NG, NSUB = DP / 64;
    constexpr uint32_t TB = L::TB;
    __shared__ __align__(8) uint64_t kvfull, qfull[NQ], qempty[NQ], gfull[NG], gempty[NG], sfull, sread, dpfull, pfull,
        done;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AttnArgs &a = t.a;

    const bool split = (int)blockIdx.x >= t.whole;
    const int share = split ? ((int)blockIdx.x - t.whole) % t.shares : 0;
    const int item = split ? t.whole + ((int)blockIdx.x - t.whole) / t.shares : blockIdx.x;
    const int kt = item % t.ktiles, hk = item / t.ktiles % a.Hkv, b = item / t.ktiles / a.Hkv;
    const int len = key_count(a, b), k0 = kt * kTile;
    const int total = t.hs_kv * t.qtiles, per = split ? t.per : total, i0 = share * per;
    const int n = k0 < len ? min(total, i0 + per) - i0 : 0;
    const int key = k0 + 32 * (warp & 3) + lane; // of warps 0-7
    if (n <= 0) { // keys behind the length: zeros (with shares, the sum writes them)
        if (!split && warp < 8 && key < a.Nk) {
            __nv_bfloat16 *dst = (warp < 4 ? a.dv : a.dk).row(b, key, hk);
            for (int d = 0; d < a.D; d += 8)
                *reinterpret_cast<uint4 *>(dst + d) = make_uint4(0, 0, 0, 0);
        }
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&kvfull), 1);
        for (int s = 0; s < NQ; ++s) {
            mbar_init(smem_addr(&qfull[s]), 1);
            mbar_init(smem_addr(&qempty[s]), 1);
        }
        for (int s = 0; s < NG; ++s) {
            mbar_init(smem_addr(&gfull[s]), 1);
            mbar_init(smem_addr(&gempty[s]), 1);
        }
        mbar_init(smem_addr(&sfull), 1);
        mbar_init(smem_addr(&dpfull), 1);
        mbar_init(smem_addr(&sread), 8);
        mbar_init(smem_addr(&pfull), 8);
        mbar_init(smem_addr(&done), 1);
        abort_s = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_addr(&tmem_base_s), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    volatile int *abort = &abort_s;
    const uint32_t s_col = tmem, dp_col = tmem + 128, dv_col = tmem + 256, dk_col = tmem + 256 + DP;

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9 && lane == 0) {
            auto load = [&](const CUtensorMap *map, uint32_t dst, uint32_t bar, int h, int row, int bb) {
                for (int s = 0; s < NSUB; ++s)
                    tma_load_4d(dst + s * SUB, map, 64 * s, h, row, bb, bar);
            };
            mbar_expect_tx(smem_addr(&kvfull), 2 * TB);
            load(&kmap, base + L::k, smem_addr(&kvfull), hk * t.kh, k0, b * t.kb);
            load(&vmap, base + L::v, smem_addr(&kvfull), hk * t.vh, k0, b * t.vb);
            int i = 0, iq = 0, ig = 0;
            for (; i < n; ++i) {
                const int set = (i0 + i) / t.qtiles, qt = (i0 + i) - set * t.qtiles, hs = hk * t.hs_kv + set;
                const int row = qt * (kTile / t.gp);
                const uint32_t qs = i % NQ, gs = i % NG;
                if (!wait_or_abort(smem_addr(&qempty[qs]), ((i / NQ) & 1u) ^ 1u, abort))
                    break;
                const uint32_t qbar = smem_addr(&qfull[qs]), st = base + L::st + qs * 1024;
                mbar_expect_tx(qbar, TB + 1024);
                load(&qmap, base + L::q + qs * TB, qbar, hs * t.gp, row, b * t.qb);
                const int64_t at = ((int64_t)b * t.hsets + hs) * t.rows + qt * kTile;
                bulk_load(st, t.lse2 + at, 512, qbar);
                bulk_load(st + 512, t.delta + at, 512, qbar);
                ++iq;
                if (!wait_or_abort(smem_addr(&gempty[gs]), ((i / NG) & 1u) ^ 1u, abort))
                    break;
                mbar_expect_tx(smem_addr(&gfull[gs]), TB);
                load(&gmap, base + L::g + gs * TB, smem_addr(&gfull[gs]), hs * t.gp, row, b * t.gb);
                ++ig;
            }
            if (i < n) { // let the copies already issued land before the CTA exits (each wait bounded)
                mbar_wait(smem_addr(&kvfull), 0u);
                for (int j = max(0, iq - NQ); j < iq; ++j)
                    mbar_wait(smem_addr(&qfull[j % NQ]), (j / NQ) & 1u);
                for (int j = max(0, ig - NG); j < ig; ++j)
                    mbar_wait(smem_addr(&gfull[j % NG]), (j / NG) & 1u);
            }
        }
        if (warp == 8 && lane == 0) {
            const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile), idesc_d = idesc_bf16_f32(kTile, DP) | kBTransposed;
            const uint64_t kd = sw128_desc(base + L::k), vd = sw128_desc(base + L::v);
            auto scores = [&](uint32_t col, uint64_t ad, uint32_t tile, uint64_t *bar) {
                const uint64_t bd = sw128_desc(tile);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    umma_bf16(col, ad + (kmajor_step(k) >> 4), bd + (kmajor_step(k) >> 4), idesc_s, k != 0);
                umma_commit(smem_addr(bar));
            };
            auto grads = [&](uint32_t col, uint32_t acol, uint32_t tile, bool add) {
                const uint64_t bd = sw128_desc_mn(tile, SUB);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k) // a warpgroup's 64 query columns: 32 packed ones
                    umma_ts(col, acol + (k / 4) * 64 + (k % 4) * 8, bd + ((k * 2048) >> 4), idesc_d, add || k > 0);
            };
            auto full = [&](uint64_t *bars, int i, int stages) {
                return wait_or_abort(smem_addr(&bars[i % stages]), (i / stages) & 1u, abort);
            };
            bool ok = wait_or_abort(smem_addr(&kvfull), 0u, abort) && full(qfull, 0, NQ);
            if (ok) {
                tc_fence_after();
                scores(s_col, kd, base + L::q, &sfull);
                ok = full(gfull, 0, NG);
            }
            if (ok) {
                tc_fence_after();
                scores(dp_col, vd, base + L::g, &dpfull);
            }
            for (int i = 0; i < n && ok; ++i) {
                if (i + 1 < n) { // s(i + 1) as soon as s(i) is in registers
                    ok = full(qfull, i + 1, NQ) && wait_or_abort(smem_addr(&sread), i & 1u, abort);
                    if (!ok)
                        break;
                    tc_fence_after();
                    scores(s_col, kd, base + L::q + ((i + 1) % NQ) * TB, &sfull);
                }
                ok = wait_or_abort(smem_addr(&pfull), i & 1u, abort);
                if (!ok)
                    break;
                tc_fence_after();
                grads(dv_col, dp_col, base + L::g + (i % NG) * TB, i > 0);
                umma_commit(smem_addr(&gempty[i % NG]));
                grads(dk_col, dp_col + 32, base + L::q + (i % NQ) * TB, i > 0);
                umma_commit(smem_addr(&qempty[i % NQ]));
                if (i + 1 < n) {
                    ok = full(gfull, i + 1, NG);
                    if (!ok)
                        break;
                    tc_fence_after();
                    scores(dp_col, vd, base + L::g + ((i + 1) % NG) * TB, &dpfull);
                }
            }
            umma_commit(smem_addr(&done));
            mbar_wait(smem_addr(&done), 0u); // every MMA issued has completed before tensor memory is freed
        }
    } else {
        regs_inc<kMathRegs>();
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t sc = s_col + lanes + 64 * half, dc = dp_col + lanes + 64 * half;
        const bool live = key < len;
        const float2 mul = make_float2(a.scale2, a.scale2);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const uint32_t qs = i % NQ;
            const float *stats = reinterpret_cast<const float *>(smem_raw + (base + L::st + qs * 1024 - smem_addr(smem_raw)));
            if (!wait_or_abort(smem_addr(&sfull), i & 1u, abort) ||
                !wait_or_abort(smem_addr(&qfull[qs]), (i / NQ) & 1u, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            float p[64];
            load_half(sc, p);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&sread));
            __syncwarp();
            // Query rows behind the last one are zeros, of which a key of -inf makes NaN: a number in its place,
            // and their lse2 of +inf, give the weight 0.  (A NaN of a query's own is in its lse2 as well.)
            if (__builtin_expect(stats[64 * half + 63] == INFINITY, 0)) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    p[e] = fmaxf(p[e], -3.402823466e+38f);
            }
            {
                const float4 *l4 = reinterpret_cast<const float4 *>(stats + 64 * half);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float4 l = l4[e];
                    const float2 x = __ffma2_rn(make_float2(p[4 * e], p[4 * e + 1]), mul, make_float2(-l.x, -l.y));
                    const float2 y = __ffma2_rn(make_float2(p[4 * e + 2], p[4 * e + 3]), mul, make_float2(-l.z, -l.w));
                    p[4 * e] = exp2_fast(x.x);
                    p[4 * e + 1] = exp2_fast(x.y);
                    p[4 * e + 2] = exp2_fast(y.x);
                    p[4 * e + 3] = exp2_fast(y.y);
                }
            }
            if (!wait_or_abort(smem_addr(&dpfull), i & 1u, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            {
                // p and ds go over this half of dp: 32 packed columns each.
                const float4 *d4 = reinterpret_cast<const float4 *>(stats + 128 + 64 * half);
                float dp[64];
                load_half(dc, dp);
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    pk[e] = live ? pack_bf16x2(p[2 * e], p[2 * e + 1]) : 0u;
                tmem_st32(dc, pk);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float4 d = d4[e];
                    const float2 x = __fmul2_rn(make_float2(p[4 * e], p[4 * e + 1]),
                                                make_float2(dp[4 * e] - d.x, dp[4 * e + 1] - d.y));
                    const float2 y = __fmul2_rn(make_float2(p[4 * e + 2], p[4 * e + 3]),
                                                make_float2(dp[4 * e + 2] - d.z, dp[4 * e + 3] - d.w));
                    pk[2 * e] = live ? pack_bf16x2(x.x, x.y) : 0u;
                    pk[2 * e + 1] = live ? pack_bf16x2(y.x, y.y) : 0u;
                }
                tmem_st32(dc + 32, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&pfull));
            __syncwarp(); // the arrival goes out before any lane begins to wait
        }
        ok = ok && wait_or_abort(smem_addr(&done), 0u, abort);
        if (ok) { // warps 0-3 store dv, 4-7 dk
            tc_fence_after();
            const uint32_t col = (half ? dk_col : dv_col) + lanes;
            const float f = half ? a.scale : 1.0f;
            float *part = t.part + ((((int64_t)share * 2 + half) * t.tail + item - t.whole) * kTile + key - k0) * a.D;
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
                uint32_t x[32];
                tmem_ld32(col + 32 * c, x);
                tmem_wait_ld();
                if (key >= a.Nk)
                    continue;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    x[e] = live ? __float_as_uint(__uint_as_float(x[e]) * f) : 0u;
#pragma unroll
                for (int e = 0; e < 2; ++e) // 16 channels
                    if (!split)
                        store16((half ? a.dk : a.dv).row(b, key, hk) + 32 * c + 16 * e, packed(x + 16 * e),
                                a.D - 32 * c - 16 * e, t.wide);
                    else
                        store16(part + 32 * c + 16 * e, x + 16 * e, a.D - 32 * c - 16 * e);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort)
        atomicAdd(&g_attn_bwd_timeouts, 1u);
}

// Without queries: dv and dk are zeros.
__global__ void __launch_bounds__(256) attn_dkv_zero_kernel(const AttnArgs a)
{
    const int64_t chunks = a.D / 8, rows = (int64_t)a.B * a.Nk * a.Hkv;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= 2 * rows * chunks)
        return;
    const int64_t half = e / (rows * chunks), r = e - half * rows * chunks, at = r / chunks;
    const int d = (int)(r - at * chunks) * 8;
    const int64_t hk = at % a.Hkv, n = at / a.Hkv;
    *reinterpret_cast<uint4 *>((half ? a.dk : a.dv).row(n / a.Nk, n % a.Nk, hk) + d) = make_uint4(0, 0, 0, 0);
}

// dv and dk of the shared tiles' partial sums, in order; zeros behind the length.
__global__ void __launch_bounds__(256) attn_dkv_sum_kernel(const BwdArgs t)
{
    const AttnArgs &a = t.a;
    const int64_t per = (int64_t)t.tail * kTile, chunks = a.D / 8;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= 2 * per * chunks)
        return;
    const int64_t half = e / (per * chunks), r = e - half * per * chunks;
    const int64_t at = r / chunks;
    const int d = (int)(r - at * chunks) * 8;
    const int item = t.whole + (int)(at / kTile);
    const int key = item % t.ktiles * kTile + (int)(at % kTile), hk = item / t.ktiles % a.Hkv, b = item / t.ktiles / a.Hkv;
    if (key >= a.Nk)
        return;
    float v[8] = {};
    if (key < key_count(a, b))
        for (int s = 0; s < t.shares; ++s) {
            float x[8];
            Row<float, 8, true>::load(t.part + ((int64_t)s * 2 + half) * per * a.D + at * a.D + d, x);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] += x[k];
        }
    Row<__nv_bfloat16, 8, true>::store((half ? a.dk : a.dv).row(b, key, hk) + d, v);
}

// dq of the shared tiles' partial sums, in order.
__global__ void __launch_bounds__(256) attn_dq_sum_kernel(const BwdArgs t)
{
    const AttnArgs &a = t.a;
    const int chunks = a.D / 8;
    const int64_t rows = (int64_t)t.dq_tail * kTile, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= rows * chunks)
        return;
    const int64_t at = e / chunks;
    const int d = (int)(e - at * chunks) * 8;
    const int item = t.dq_whole + (int)(at / kTile);
    const int row = item % t.qtiles * kTile + (int)(at % kTile), hs = item / t.qtiles % t.hsets, b = item / t.qtiles / t.hsets;
    const int iq = row / t.gp, h = hs * t.gp + row % t.gp;
    if (iq >= a.Nq)
        return;
    const int tiles = (key_count(a, b) + kTile - 1) / kTile, live = (tiles + t.dq_per - 1) / t.dq_per;
    float v[8] = {};
    for (int s = 0; s < live; ++s) {
        float x[8];
        Row<float, 8, true>::load(t.dq_part + (s * rows + at) * a.D + d, x);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] += x[k];
    }
    Row<__nv_bfloat16, 8, true>::store(a.dq.row(b, iq, h) + d, v);
}

template <int DP> struct DqSmem {
    static constexpr int NQ = DP == 128 ? 1 : 2;                         // stages of q and go,
    static constexpr int NK = DP == 128 ? 3 : 4, NV = DP == 128 ? 2 : 4; // of k and v
    static constexpr uint32_t TB = tile_bytes<DP>();
    static constexpr uint32_t q = 0, g = TB, k = 2 * NQ * TB, v = k + NK * TB; // (q and go of a stage side by side)
    static constexpr size_t bytes = v + NV * TB + 1024;
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_dq_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap gmap,
               const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const BwdArgs t)
{
    using L = DqSmem<DP>;
    constexpr int NQ = L::NQ, NK = L::NK, NV = L::NV, NSUB = DP / 64;
    constexpr uint32_t TB = L::TB;
    __shared__ __align__(8) uint64_t qfull[NQ], qempty[NQ], kfull[NK], kempty[NK], vfull[NV], vempty[NV], sfull[2], dpfull, dsfull,
        dqfull, xfull[4], drain;
    __shared__ float row_sum[2][kTile];
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AttnArgs &a = t.a;
    // Item i: query tile qt of head set hs of batch entry b, over key tiles [j0, j0 + n); of a shared tile,
    // its index among these (else -1) and the share.
    struct Item {
        int b, hs, qt, part, share, len, tiles, j0, n;
    };
    auto decode = [&](int i) {
        Item w;
        w.part = -1;
        w.share = 0;
        int r = i;
        if (i >= t.dq_whole) {
            w.part = (i - t.dq_whole) / t.dq_shares;
            w.share = (i - t.dq_whole) - w.part * t.dq_shares;
            r = t.dq_whole + w.part;
        }
        const int sets = t.qtiles_div.div(r);
        w.qt = r - sets * t.qtiles;
        w.b = t.hsets_div.div(sets);
        w.hs = sets - w.b * t.hsets;
        w.len = key_count(a, w.b);
        w.tiles = (w.len + kTile - 1) / kTile;
        w.j0 = min(w.tiles, w.share * t.dq_per);
        w.n = (w.part < 0 ? w.tiles : min(w.tiles, w.j0 + t.dq_per)) - w.j0;
        return w;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NQ; ++s) {
            mbar_init(smem_addr(&qfull[s]), 1);
            mbar_init(smem_addr(&qempty[s]), 1);
        }
        for (uint64_t *bar : {&sfull[0], &sfull[1], &dpfull, &dqfull, &drain})
            mbar_init(smem_addr(bar), 1);
        mbar_init(smem_addr(&dsfull), 8);
        for (int i = 0; i < 4; ++i)
            mbar_init(smem_addr(&xfull[i]), 2);
        for (int s = 0; s < NK; ++s) {
            mbar_init(smem_addr(&kfull[s]), 1);
            mbar_init(smem_addr(&kempty[s]), 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(smem_addr(&vfull[s]), 1);
            mbar_init(smem_addr(&vempty[s]), 1);
        }
        abort_s = 0;
        fence_barrier_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_addr(&tmem_base_s), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    volatile int *abort = &abort_s;
    const uint32_t s_col = tmem, dp_col = tmem + 256, dq_col = tmem + 384; // s: two buffers

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9 && lane == 0) {
            uint32_t ik = 0, iv = 0, iq = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap *map, uint32_t dst, uint32_t bar, int h, int row, int bb) {
                for (int s = 0; s < NSUB; ++s)
                    tma_load_4d(dst + s * SUB, map, 64 * s, h, row, bb, bar);
            };
            for (int i = blockIdx.x; i < t.dq_items && ok; i += gridDim.x) {
                const Item w = decode(i);
                const int b = w.b, hs = w.hs, qt = w.qt, n = w.n, hk = hs / t.hs_kv;
                if (n == 0)
                    continue;
                const uint32_t qs = iq % NQ, at = base + qs * 2 * TB, qbar = smem_addr(&qfull[qs]);
                ok = wait_or_abort(smem_addr(&qempty[qs]), ((iq / NQ) & 1u) ^ 1u, abort);
                if (!ok)
                    break;
                mbar_expect_tx(qbar, 2 * TB);
                load(&qmap, at + L::q, qbar, hs * t.gp, qt * (kTile / t.gp), b * t.qb);
                load(&gmap, at + L::g, qbar, hs * t.gp, qt * (kTile / t.gp), b * t.gb);
                ++iq;
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t ks = ik % NK, vs = iv % NV;
                    ok = wait_or_abort(smem_addr(&kempty[ks]), ((ik / NK) & 1u) ^ 1u, abort);
                    if (!ok)
                        break;
                    mbar_expect_tx(smem_addr(&kfull[ks]), TB);
                    load(&kmap, base + L::k + ks * TB, smem_addr(&kfull[ks]), hk * t.kh, (w.j0 + j) * kTile, b * t.kb);
                    ++ik;
                    ok = wait_or_abort(smem_addr(&vempty[vs]), ((iv / NV) & 1u) ^ 1u, abort);
                    if (!ok)
                        break;
                    mbar_expect_tx(smem_addr(&vfull[vs]), TB);
                    load(&vmap, base + L::v + vs * TB, smem_addr(&vfull[vs]), hk * t.vh, (w.j0 + j) * kTile, b * t.vb);
                    ++iv;
                }
            }
            if (!ok) { // let the copies already issued land before the CTA exits (each wait bounded)
                for (uint32_t j = iq > (uint32_t)NQ ? iq - NQ : 0; j < iq; ++j)
                    mbar_wait(smem_addr(&qfull[j % NQ]), (j / NQ) & 1u);
                for (uint32_t j = ik > (uint32_t)NK ? ik - NK : 0; j < ik; ++j)
                    mbar_wait(smem_addr(&kfull[j % NK]), (j / NK) & 1u);
                for (uint32_t j = iv > (uint32_t)NV ? iv - NV : 0; j < iv; ++j)
                    mbar_wait(smem_addr(&vfull[j % NV]), (j / NV) & 1u);
            }
        }
        if (warp == 8 && lane == 0) {
            const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile), idesc_d = idesc_bf16_f32(kTile, DP) | kBTransposed;
            const uint64_t qd = sw128_desc(base + L::q), gd = sw128_desc(base + L::g);
            uint32_t it = 0, iq = 0; // key tiles, items so far
            bool ok = true;
            auto product = [&](uint32_t col, uint64_t ad, uint32_t tile) {
                const uint64_t bd = sw128_desc(tile);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    umma_bf16(col, ad + (kmajor_step(k) >> 4), bd + (kmajor_step(k) >> 4), idesc_s, k != 0);
            };
            auto scores = [&](uint32_t x, uint32_t m) { // s of key tile x (counted over all items) for item m
                if (!wait_or_abort(smem_addr(&kfull[x % NK]), (x / NK) & 1u, abort))
                    return false;
                tc_fence_after();
                product(s_col + 128 * (x & 1u), qd + ((m % NQ * 2 * TB) >> 4), base + L::k + (x % NK) * TB);
                umma_commit(smem_addr(&sfull[x & 1u]));
                return true;
            };
            auto first = [&](uint32_t x, uint32_t m) {
                return wait_or_abort(smem_addr(&qfull[m % NQ]), (m / NQ) & 1u, abort) && scores(x, m);
            };
            auto dps = [&](uint32_t x, uint32_t m) {
                if (!wait_or_abort(smem_addr(&vfull[x % NV]), (x / NV) & 1u, abort))
                    return false;
                tc_fence_after();
                product(dp_col, gd + ((m % NQ * 2 * TB) >> 4), base + L::v + (x % NV) * TB);
                umma_commit(smem_addr(&dpfull));
                umma_commit(smem_addr(&vempty[x % NV]));
                return true;
            };
            // The item after i that has keys: its number of key tiles (0: there is none).
            auto next = [&](int &i) {
                for (i += gridDim.x; i < t.dq_items; i += gridDim.x) {
                    const int n = decode(i).n;
                    if (n)
                        return n;
                }
                return 0;
            };
            int i = (int)blockIdx.x - (int)gridDim.x, n = next(i);
            ok = n == 0 || first(0, 0);
            while (n && ok) { // the first scores of the item have been issued
                const int n2 = next(i);
                ok = dps(it, iq) && (n == 1 || scores(it + 1, iq));
                if (n == 1 && ok)
                    umma_commit(smem_addr(&qempty[iq % NQ]));
                for (int j = 0; j < n && ok; ++j) {
                    const uint32_t x = it + j;
                    // With two stages of q: the next item's first scores under this item's last arithmetic.
                    if (NQ == 2 && j + 1 == n && n2 && !first(x + 1, iq + 1)) {
                        ok = false;
                        break;
                    }
                    ok = wait_or_abort(smem_addr(&dsfull), x & 1u, abort);
                    if (!ok)
                        break;
                    tc_fence_after();
                    const uint64_t bd = sw128_desc_mn(base + L::k + (x % NK) * TB, SUB);
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k) // a warpgroup's 64 key columns: 32 packed ones
                        umma_ts(dq_col, s_col + 128 * (x & 1u) + (k / 4) * 64 + (k % 4) * 8, bd + ((k * 2048) >> 4),
                                idesc_d, j > 0 || k > 0);
                    umma_commit(smem_addr(&kempty[x % NK]));
                    if (j + 1 < n) {
                        ok = dps(x + 1, iq) && (j + 2 >= n || scores(x + 2, iq));
                        if (j + 2 == n && ok)
                            umma_commit(smem_addr(&qempty[iq % NQ]));
                    } else
                        umma_commit(smem_addr(&dqfull));
                }
                it += n;
                ++iq;
                if (NQ == 1 && n2 && ok)
                    ok = first(it, iq);
                n = n2;
            }
            umma_commit(smem_addr(&drain));
            mbar_wait(smem_addr(&drain), 0u); // every MMA issued has completed before tensor memory is freed
        }
    } else {
        regs_inc<kMathRegs>();
        const int half = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const float2 mul = make_float2(a.scale2, a.scale2);
        uint32_t it = 0, items = 0, nx = 0;
        bool ok = true;
        auto stat_at = [&](const Item &w) {
            return ((int64_t)w.b * t.hsets + w.hs) * t.rows + w.qt * kTile + 32 * (warp & 3) + lane;
        };
        Item w = decode(min((int)blockIdx.x, t.dq_items - 1));
        float lse2 = t.lse2[stat_at(w)], delta = t.delta[stat_at(w)];
        for (int i = blockIdx.x; i < t.dq_items && ok; i += gridDim.x) {
            const int b = w.b, hs = w.hs, qt = w.qt, len = w.len, n = w.n;
            const int row = qt * kTile + 32 * (warp & 3) + lane;
            const int iq = row >> t.lgp, h = hs * t.gp + (row & (t.gp - 1));
            const int64_t at = stat_at(w);
            const float2 l2 = make_float2(-lse2, -lse2);
            for (int j = 0; j < n; ++j, ++it) {
                const uint32_t sc = s_col + 128 * (it & 1u) + 64 * half + lanes;
                if (!wait_or_abort(smem_addr(&sfull[it & 1u]), (it >> 1) & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float p[64];
                load_half(sc, p);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 x = __ffma2_rn(make_float2(p[2 * e], p[2 * e + 1]), mul, l2);
                    p[2 * e] = exp2_fast(x.x);
                    p[2 * e + 1] = exp2_fast(x.y);
                }
                if (!wait_or_abort(smem_addr(&dpfull), it & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int valid = len - (w.j0 + j) * kTile; // keys of this tile
                {
                    float dp[64];
                    load_half(dp_col + 64 * half + lanes, dp);
                    if (w.tiles == 1) { // all keys are here: delta = sum p dp, for attn_dkv_kernel as well
                        float sum[4] = {};
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            sum[e & 3] += 64 * half + e < valid ? p[e] * dp[e] : 0.0f;
                        const int lrow = 32 * (warp & 3) + lane;
                        row_sum[half][lrow] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(smem_addr(&xfull[warp & 3]));
                        __syncwarp();
                        if (!wait_or_abort(smem_addr(&xfull[warp & 3]), nx++ & 1u, abort)) {
                            ok = false;
                            break;
                        }
                        delta = row_sum[0][lrow] + row_sum[1][lrow];
                        if (half == 0 && iq < a.Nq) // (0 behind the last row)
                            t.delta[at] = delta;
                    }
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 x = __fmul2_rn(make_float2(p[2 * e], p[2 * e + 1]),
                                                    make_float2(dp[2 * e] - delta, dp[2 * e + 1] - delta));
                        pk[e] = pack_bf16x2(x.x, x.y);
                    }
                    if (valid < kTile) { // keys behind the length: 0, whatever their scores
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int c = 64 * half + 2 * e;
                            pk[e] = c + 1 < valid ? pk[e] : c < valid ? pk[e] & 0xFFFFu : 0u;
                        }
                    }
                    tmem_st32(sc, pk);
                }
                if (half == 0 && valid < kTile && len < a.Nk) { // and the k rows themselves
                    const uint32_t ks = it % NK;
                    if (!wait_or_abort(smem_addr(&kfull[ks]), (it / NK) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    unsigned char *k = smem_raw + (base + L::k + ks * TB - smem_addr(smem_raw));
                    for (int e = valid * 8 + threadIdx.x; e < kTile * 8; e += 128)
#pragma unroll
                        for (int sub = 0; sub < NSUB; ++sub)
                            *reinterpret_cast<uint4 *>(k + sub * SUB + e * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&dsfull));
                __syncwarp(); // the arrival goes out before any lane begins to wait
            }
            if (!ok)
                break;
            // The next item's statistics are on their way while this one's products end.
            const Item done = w;
            if (i + gridDim.x < t.dq_items) {
                w = decode(i + gridDim.x);
                lse2 = t.lse2[stat_at(w)];
                delta = t.delta[stat_at(w)];
            }
            if (n > 0) {
                if (!wait_or_abort(smem_addr(&dqfull), items & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                ++items;
            }
            // Each warpgroup stores half of the channels; with shares, the partial sum.
            float *part = t.dq_part + (((int64_t)done.share * t.dq_tail + done.part) * kTile + row - qt * kTile) * a.D;
#pragma unroll
            for (int c = 0; c < DP / 64; ++c) {
                uint32_t x[32] = {};
                const int d0 = half * (DP / 2) + 32 * c;
                if (n > 0) {
                    tmem_ld32(dq_col + d0 + lanes, x);
                    tmem_wait_ld();
                }
                if (iq >= a.Nq || (done.part >= 0 && n == 0)) // (a share without keys is not read)
                    continue;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    x[e] = n > 0 ? __float_as_uint(__uint_as_float(x[e]) * a.scale) : 0u;
#pragma unroll
                for (int e = 0; e < 2; ++e) // 16 channels
                    if (done.part < 0)
                        store16(a.dq.row(b, iq, h) + d0 + 16 * e, packed(x + 16 * e), a.D - d0 - 16 * e, t.dq_wide);
                    else
                        store16(part + d0 + 16 * e, x + 16 * e, a.D - d0 - 16 * e);
            }
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort)
        atomicAdd(&g_attn_bwd_timeouts, 1u);
}

template <typename K> tok_status prepare(K kernel, size_t smem)
{
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    return TOK_OK;
}

template <int DP> tok_status launch(const BwdArgs &t, const CUtensorMap &q, const CUtensorMap &g, const CUtensorMap &k,
                                    const CUtensorMap &v, cudaStream_t stream)
{
    const AttnArgs &a = t.a;
    tok_status st = prepare(attn_dkv_kernel<DP>, DkvSmem<DP>::bytes);
    if (st == TOK_OK)
        st = prepare(attn_dq_kernel<DP>, DqSmem<DP>::bytes);
    if (st != TOK_OK)
        return st;
    const int sms = sm_count();
    attn_dq_kernel<DP><<<std::min(t.dq_items, sms > 0 ? sms : 1), kThreads, DqSmem<DP>::bytes, stream>>>(q, g, k, v, t);
    st = launch_status();
    if (st == TOK_OK && t.dq_tail > 0) {
        const int64_t threads = (int64_t)t.dq_tail * kTile * (a.D / 8);
        attn_dq_sum_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(t);
        st = launch_status();
    }
    if (st == TOK_OK && t.ktiles > 0) {
        attn_dkv_kernel<DP><<<(unsigned)(t.whole + t.tail * t.shares), kThreads, DkvSmem<DP>::bytes, stream>>>(
            q, g, k, v, t);
        st = launch_status();
    }
    return st;
}

// Tiles and shares of a backward call, from its extents alone.
struct Plan {
    int64_t gp, hsets, qtiles, rows, ktiles, hs_kv, stat_floats;
    int64_t whole, tail, shares, per, part_floats;
    int64_t dq_whole, dq_tail, dq_shares, dq_per, dq_floats;
    Plan(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D)
    {
        gp = attn_tc_group((int)(Hq / Hkv));
        hsets = Hq / gp;
        hs_kv = hsets / Hkv;
        qtiles = (Nq * gp + kTile - 1) / kTile;
        rows = qtiles * kTile;
        ktiles = (Nk + kTile - 1) / kTile;
        stat_floats = B * hsets * rows;
        // Shares of the query tiles: the least of an estimate in us.  A share costs its tiles (1.8 us each,
        // 1.6 with narrow heads) and 5 us around them; the last round of the SMs is half full on
        // average (batch entries end early); partial sums are written and read once.  (2 x 28
        // tiles of 3520 keys, 16 heads: 1 share, 2 cost 60 us more; 4 x 4 tiles of 512 ragged
        // keys over 220 query tiles: 8, against 1.8 times as long with 1.)
        const int64_t total = hs_kv * qtiles, base = B * Hkv * ktiles;
        const double tile_us = D > 64 ? 1.8 : 1.6, part_us = 2.0 * kTile * 4 * D / 6.0e6;
        whole = base;
        tail = 0;
        shares = 1;
        per = std::max<int64_t>(1, total);
        double best = 0;
        for (int64_t s = 1; base > 0 && s <= 16 && s <= std::max<int64_t>(1, total / 4); ++s) {
            const double rounds = std::max(1.0, (double)(base * s) / 148 + 0.5);
            const double us = rounds * ((double)((total + s - 1) / s) * tile_us + 5) +
                              (s > 1 ? 4 + (double)(s * base) * 2 * part_us : 0);
            if (s == 1 || us < best) {
                best = us;
                shares = s;
            }
        }
        if (shares > 1) {
            whole = 0;
            tail = base;
            per = (total + shares - 1) / shares;
            shares = (total + per - 1) / per;
        } else if (base > 148) { // one each pays; the last round's may be shared all the same
            const Rounds r(base, total, 16, tile_us, 5, 2 * part_us);
            whole = r.whole;
            tail = r.tail;
            shares = r.shares;
            per = r.per;
        }
        part_floats = tail * shares * 2 * kTile * D;
        const Rounds r(B * hsets * qtiles, ktiles, 32, 1.6, 4, part_us);
        dq_whole = r.whole;
        dq_tail = r.tail;
        dq_shares = r.shares;
        dq_per = r.per;
        dq_floats = dq_tail * dq_shares * kTile * D;
    }
};

} // namespace

int64_t attn_tc_backward_workspace(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D)
{
    const Plan p(B, Nq, Nk, Hq, Hkv, D);
    return (2 * p.stat_floats + p.part_floats + p.dq_floats) * 4;
}

tok_status attn_tc_backward(const AttnArgs &a, float *workspace, cudaStream_t stream)
{
    const Plan p(a.B, a.Nq, a.Nk, a.Hq, a.Hkv, a.D);
    BwdArgs t{};
    t.a = a;
    t.lse2 = workspace;
    t.delta = workspace + p.stat_floats;
    t.part = workspace + 2 * p.stat_floats;
    t.dq_part = t.part + p.part_floats;
    t.dq_whole = (int)p.dq_whole;
    t.dq_tail = (int)p.dq_tail;
    t.dq_items = (int)(p.dq_whole + p.dq_tail * p.dq_shares);
    t.dq_shares = (int)p.dq_shares;
    t.dq_per = (int)p.dq_per;
    t.gp = (int)p.gp;
    while (t.gp >> t.lgp > 1)
        ++t.lgp;
    t.hsets = (int)p.hsets;
    t.qtiles_div = FastDiv((uint32_t)std::max<int64_t>(1, p.qtiles));
    t.hsets_div = FastDiv((uint32_t)p.hsets);
    t.dq_wide = rows_wide(a.dq, a.B, a.Nq, a.Hq);
    t.wide = rows_wide(a.dk, a.B, a.Nk, a.Hkv) && rows_wide(a.dv, a.B, a.Nk, a.Hkv);
    t.rows = (int)p.rows;
    t.qtiles = (int)p.qtiles;
    t.ktiles = (int)p.ktiles;
    t.hs_kv = (int)p.hs_kv;
    t.whole = (int)p.whole;
    t.tail = (int)p.tail;
    t.shares = (int)p.shares;
    t.per = (int)p.per;
    t.qb = a.B > 1 && a.q.b == 0 ? 0 : 1;
    t.gb = a.B > 1 && a.go.b == 0 ? 0 : 1;
    t.kb = a.B > 1 && a.k.b == 0 ? 0 : 1;
    t.vb = a.B > 1 && a.v.b == 0 ? 0 : 1;
    t.kh = a.Hkv > 1 && a.k.h == 0 ? 0 : 1;
    t.vh = a.Hkv > 1 && a.v.h == 0 ? 0 : 1;
    tok_status st = TOK_OK;
    if (a.Nq > 0) {
        const auto stats = a.D <= 64 ? attn_stats_kernel<64> : attn_stats_kernel<128>;
        stats<<<(unsigned)(p.stat_floats / kTile), 256, 0, stream>>>(t, workspace, workspace + p.stat_floats);
        st = launch_status();
    }
    if (st == TOK_OK && a.Nq > 0) {
        // Without keys the maps of k and v stand on q: no kernel reads through them.
        const bool keys = a.Nk > 0;
        const HeadsView none{a.q.p, 0, 0, 0};
        CUtensorMap q, g, k, v;
        const int qr = kTile / t.gp;
        if (!heads_map(&q, a.q, a.B, a.Nq, a.Hq, a.D, t.gp, qr) || !heads_map(&g, a.go, a.B, a.Nq, a.Hq, a.D, t.gp, qr) ||
            !(keys ? heads_map(&k, a.k, a.B, a.Nk, a.Hkv, a.D, 1, kTile) : heads_map(&k, none, 1, 1, 1, a.D, 1, kTile)) ||
            !(keys ? heads_map(&v, a.v, a.B, a.Nk, a.Hkv, a.D, 1, kTile) : heads_map(&v, none, 1, 1, 1, a.D, 1, kTile)))
            return TOK_ERR_SHAPE;
        st = a.D <= 64 ? launch<64>(t, q, g, k, v, stream) : launch<128>(t, q, g, k, v, stream);
    }
    if (a.Nq == 0) {
        const int64_t threads = (int64_t)a.B * a.Nk * a.Hkv * 2 * (a.D / 8);
        attn_dkv_zero_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, stream>>>(a);
        return launch_status();
    }
    if (st == TOK_OK && t.tail > 0) {
        const int64_t sum_threads = (int64_t)t.tail * kTile * 2 * (a.D / 8);
        attn_dkv_sum_kernel<<<(unsigned)((sum_threads + 255) / 256), 256, 0, stream>>>(t);
        st = launch_status();
    }
    return st;
}

tok_status read_and_clear_attn_bwd_timeouts(cudaStream_t stream, unsigned int *count)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_attn_bwd_timeouts, sizeof(unsigned int), 0,
                                              cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && *count)
        e = cudaMemcpyToSymbolAsync(g_attn_bwd_timeouts, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    return TOK_OK;
}

} // namespace tok
