// Cross attention forward on the 5th-generation tensor cores, for calls with enough query
// rows to fill their 128-row tiles.
//
// A work item is 256 query rows of one key head (two tiles of 128) against the item's share
// of the keys, in tiles of 128.  Where the query heads of a group are a power of two, a tile
// holds 128 / G tokens x G heads, so a group reads its keys once.  One CTA per SM walks the
// items; its warps:
//   warps 0-3, 4-7  softmax of row tile 0 / 1, one thread per row (its lane of tensor
//                   memory): scores -> running maximum and sum -> weights, rounded to
//                   bf16, back into the scores' columns as the A operand of the second
//                   product; at the end o / sum -> HBM.  The accumulator is rescaled only
//                   when the maximum has grown by more than 2^8 (every term carries the
//                   same factor, so the quotient is unchanged; 2^8 is far from overflow).
//   warp 8          one thread issues the MMAs: o_i += p_i v_j, then s_i = q_i k_(j+1) (of the next
//                   item where j was the last), for i = 0, 1 in turn, so that one tile's MMAs run
//                   under the other's softmax and an item's first scores under the stores of the one before;
//   warp 9          tensor copies of q, k, v into 128-byte-swizzled tiles (zero-filled
//                   past the tensor: D below the tile's width needs no other care).
// What bounds it: the 16 exponentials an SM takes per cycle (1,024 cycles for a tile of scores) and the chain
// scores -> softmax -> product of a row tile, which two row tiles in turn do not hide in full.  Measured, 16
// heads of 128: 56,320 queries x 512 keys 249 us (947 TFLOP/s), 14,080 x 2048 203 us; of 64: 213
// and 179 us.  Rows of o go straight from registers to HBM, one per thread, in 32-byte sectors: through a
// staging buffer and tensor stores an item of one key tile took 7% (64 channels) longer.
// The v rows behind a batch entry's length are zeroed in shared memory (a weight of 0 times
// NaN would be NaN); scores behind it are -inf.  All waits are bounded as in the convolutions.
#include <algorithm>

#include "attention.cuh"

namespace tok {

static __device__ unsigned int g_attn_timeouts = 0;

namespace {

constexpr int kTile = 128;
constexpr int kThreads = 384; // warps 10 and 11 only make the register split whole
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88; // 256 x 208 + 128 x 88 = 384 x 168 at launch
constexpr float kGrow = 8.0f; // log2 of the growth of the maximum that the weights absorb

template <int DP> constexpr uint32_t tile_bytes() { return kTile * DP * 2; }
template <int DP> constexpr int stages() { return DP == 128 ? 4 : 8; }
template <int DP> constexpr size_t smem_bytes()
{
    return (2 + stages<DP>()) * (size_t)tile_bytes<DP>() + 1024;
}

struct TcArgs {
    AttnArgs a;
    int gp, lgp;  // heads of a row tile (a power of two)
    int wide;     // rows of o start on 32 bytes
    int nqt;      // items per (batch, head set): 256 rows each
    int hsets;    // Hq / gp
    FastDiv nqt_div, hsets_div;
    int items;    // CTAs' worth: whole ones, then the shares of the others
    int whole, tail;
    int qb, kb, kh, vb, vh; // coordinate factors: 0 for a broadcast dimension
};

struct Item {
    int b, hs, row0, k0, ntiles, kend, split, part; // part: index among the split items, or -1
};

__device__ __forceinline__ void place(const TcArgs &t, int r, Item &w)
{
    const int sets = t.nqt_div.div(r);
    w.row0 = (r - sets * t.nqt) * (2 * kTile);
    w.b = t.hsets_div.div(sets);
    w.hs = sets - w.b * t.hsets;
}

__device__ __forceinline__ Item decode(const TcArgs &t, int i)
{
    Item w;
    int splits = 1;
    w.split = 0;
    w.part = -1;
    if (i >= t.whole) {
        splits = t.a.splits;
        w.part = (i - t.whole) / splits;
        w.split = (i - t.whole) - w.part * splits;
        i = t.whole + w.part;
    }
    place(t, i, w);
    const int len = key_count(t.a, w.b), tiles = (len + kTile - 1) / kTile;
    const int per = (tiles + splits - 1) / splits;
    const int t0 = min(tiles, w.split * per), t1 = min(tiles, t0 + per);
    w.k0 = t0 * kTile;
    w.ntiles = t1 - t0;
    w.kend = min(len, t1 * kTile);
    return w;
}

// Row of a split item in the partial results, and these' statistics (maximum, sum).
__device__ __forceinline__ int64_t part_row(const TcArgs &t, const Item &w, int row)
{
    return ((int64_t)w.split * t.tail + w.part) * (2 * kTile) + (row - w.row0);
}
__device__ __forceinline__ float2 *part_stats(const TcArgs &t)
{
    return reinterpret_cast<float2 *>(t.a.part + (int64_t)t.a.splits * t.tail * (2 * kTile) * t.a.D);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
attn_fwd_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const TcArgs t)
{
    constexpr int NST = stages<DP>(), NSUB = DP / 64;
    constexpr uint32_t TB = tile_bytes<DP>(), SUB = kTile * 128;
    __shared__ __align__(8) uint64_t qfull[2], qempty[2], kvfull[NST], kvempty[NST], sfull[2], pfull[2], ofull[2], drain;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t kvbase = base + 2 * TB;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const AttnArgs &a = t.a;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&qfull[i]), 1);
            mbar_init(smem_addr(&qempty[i]), 1);
            mbar_init(smem_addr(&sfull[i]), 1);
            mbar_init(smem_addr(&pfull[i]), 4);
            mbar_init(smem_addr(&ofull[i]), 1);
        }
        for (int s = 0; s < NST; ++s) {
            mbar_init(smem_addr(&kvfull[s]), 1);
            mbar_init(smem_addr(&kvempty[s]), 1);
        }
        mbar_init(smem_addr(&drain), 1);
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
    const uint32_t s_col[2] = {tmem, tmem + 128}, o_col[2] = {tmem + 256, tmem + 256 + DP};

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 9 && lane == 0) {
            uint32_t it = 0, nq = 0, issued[2] = {0, 0};
            bool ok = true;
            auto load = [&](const CUtensorMap *map, uint32_t dst, uint32_t bar, int h, int n, int b) {
                mbar_expect_tx(bar, TB);
                for (int s = 0; s < NSUB; ++s)
                    tma_load_4d(dst + s * SUB, map, 64 * s, h, n, b, bar);
            };
            auto load_q = [&](const Item &w, int i) {
                if (!wait_or_abort(smem_addr(&qempty[i]), (nq & 1u) ^ 1u, abort))
                    return false;
                load(&qmap, base + i * TB, smem_addr(&qfull[i]), w.hs * t.gp, (w.row0 + i * kTile) >> t.lgp,
                     w.b * t.qb);
                ++issued[i];
                return true;
            };
            auto load_kv = [&](const Item &w, int j, bool v) {
                const uint32_t s = it % NST;
                if (!wait_or_abort(smem_addr(&kvempty[s]), ((it / NST) & 1u) ^ 1u, abort))
                    return false;
                const int hk = w.hs * t.gp / a.G;
                load(v ? &vmap : &kmap, kvbase + s * TB, smem_addr(&kvfull[s]), hk * (v ? t.vh : t.kh),
                     w.k0 + j * kTile, w.b * (v ? t.vb : t.kb));
                ++it;
                return true;
            };
            for (int i = blockIdx.x; i < t.items && ok; i += gridDim.x) {
                const Item w = decode(t, i);
                if (w.ntiles == 0)
                    continue;
                ok = load_q(w, 0) && load_kv(w, 0, false) && load_q(w, 1) && load_kv(w, 0, true);
                for (int j = 1; j < w.ntiles && ok; ++j)
                    ok = load_kv(w, j, false) && load_kv(w, j, true);
                ++nq;
            }
            if (!ok) { // let the copies already issued land before the CTA exits (each wait bounded)
                for (uint32_t j = it > (uint32_t)NST ? it - NST : 0; j < it; ++j)
                    mbar_wait(smem_addr(&kvfull[j % NST]), (j / NST) & 1u);
                for (int i = 0; i < 2; ++i)
                    if (issued[i])
                        mbar_wait(smem_addr(&qfull[i]), (issued[i] - 1) & 1u);
            }
        }
        if (warp == 8 && lane == 0) {
            const uint32_t idesc_s = idesc_bf16_f32(kTile, kTile), idesc_o = idesc_bf16_f32(kTile, DP) | kBTransposed;
            const uint64_t qdesc = sw128_desc(base), kdesc = sw128_desc(kvbase);
            const uint64_t vdesc = sw128_desc_mn(kvbase, SUB);
            uint32_t it = 0, nq = 0, np = 0; // ring position, items, key tiles (phases of pfull)
            bool ok = true;
            auto scores = [&](int i, uint32_t s) { // s_i = q_i k^T
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t off = ((k / 4) * SUB + (k % 4) * 32) >> 4;
                    umma_bf16(s_col[i], qdesc + ((i * TB) >> 4) + off, kdesc + ((s * TB) >> 4) + off, idesc_s, k != 0);
                }
                umma_commit(smem_addr(&sfull[i]));
            };
            // The item after i that has keys: its number of key tiles (0: there is none).
            auto next = [&](int &i) {
                for (i += gridDim.x; i < t.items; i += gridDim.x) {
                    const int n = decode(t, i).ntiles;
                    if (n)
                        return n;
                }
                return 0;
            };
            int i = (int)blockIdx.x - (int)gridDim.x, n = next(i);
            if (n) { // the first scores; those of a later item follow the last products of the one before
                ok = wait_or_abort(smem_addr(&kvfull[0]), 0u, abort);
                for (int r = 0; r < 2 && ok; ++r) {
                    ok = wait_or_abort(smem_addr(&qfull[r]), 0u, abort);
                    if (!ok)
                        break;
                    tc_fence_after();
                    scores(r, 0);
                    if (n == 1)
                        umma_commit(smem_addr(&qempty[r]));
                }
                if (ok)
                    umma_commit(smem_addr(&kvempty[0]));
                it = nq = 1;
            }
            while (n && ok) {
                const int n2 = next(i);
                for (int j = 0; j < n && ok; ++j, ++np, it += 2) {
                    const bool last = j + 1 == n, more = !last || n2;
                    const uint32_t vs = it % NST, kn = (it + 1) % NST;
                    ok = wait_or_abort(smem_addr(&kvfull[vs]), (it / NST) & 1u, abort) &&
                         (!more || wait_or_abort(smem_addr(&kvfull[kn]), ((it + 1) / NST) & 1u, abort));
                    for (int r = 0; r < 2 && ok; ++r) {
                        ok = wait_or_abort(smem_addr(&pfull[r]), np & 1u, abort);
                        if (!ok)
                            break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            umma_ts(o_col[r], s_col[r] + 8 * k, vdesc + ((vs * TB + k * 2048) >> 4), idesc_o,
                                    j > 0 || k > 0);
                        if (r == 1)
                            umma_commit(smem_addr(&kvempty[vs]));
                        if (last)
                            umma_commit(smem_addr(&ofull[r]));
                        if (!more)
                            continue;
                        if (last) {
                            ok = wait_or_abort(smem_addr(&qfull[r]), nq & 1u, abort);
                            if (!ok)
                                break;
                            tc_fence_after();
                        }
                        scores(r, kn);
                        if (last ? n2 == 1 : j + 2 == n)
                            umma_commit(smem_addr(&qempty[r]));
                    }
                    if (ok && more)
                        umma_commit(smem_addr(&kvempty[kn]));
                }
                ++nq;
                n = n2;
            }
            // Every MMA issued has completed before tensor memory is freed.
            umma_commit(smem_addr(&drain));
            mbar_wait(smem_addr(&drain), 0u);
        }
    } else {
        regs_inc<kSoftmaxRegs>();
        const int r = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t sc = s_col[r] + lanes, oc = o_col[r] + lanes;
        const bool odd_scale = !(a.scale2 > 0.0f);
        const float mul = odd_scale ? 1.0f : a.scale2;
        uint32_t it = 0, ns = 0, nitem = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < t.items && ok; i += gridDim.x) {
            const Item w = decode(t, i);
            const int row = w.row0 + r * kTile + 32 * (warp & 3) + lane;
            const int iq = row >> t.lgp, h = w.hs * t.gp + (row & (t.gp - 1));
            const bool live = iq < a.Nq;
            const int64_t stat = ((int64_t)w.b * a.Hq + h) * a.Nq + iq;
            float m = -INFINITY, l = 0.0f; // maximum (log2 units) that the weights are relative to; their sum
            for (int j = 0; j < w.ntiles; ++j, ++ns) {
                if (!wait_or_abort(smem_addr(&sfull[r]), ns & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                float s[kTile];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32(sc + 32 * c, reinterpret_cast<uint32_t(&)[32]>(s[32 * c]));
                tmem_wait_ld();
                if (__builtin_expect(odd_scale, 0)) { // (the seldom taken blocks out of the loop's code)
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        s[c] *= a.scale2;
                }
                const int valid = w.kend - (w.k0 + j * kTile);
                if (__builtin_expect(valid < kTile, 0)) {
#pragma unroll
                    for (int c = 0; c < kTile; ++c)
                        s[c] = c < valid ? s[c] : -INFINITY;
                }
                float mx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    mx[e] = s[e];
#pragma unroll
                for (int c = 8; c < kTile - 8; c += 16) // (two new values to a three-operand maximum)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        mx[e] = fmaxf(fmaxf(mx[e], s[c + e]), s[c + 8 + e]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    mx[e] = fmaxf(mx[e], s[kTile - 8 + e]);
                const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                        fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * mul;
                if (j == 0)
                    m = fmaxf(top, -3.402823466e+38f); // (where every score is -inf, any later one moves it)
                else {
                    const bool grow = top > m + kGrow;
                    if (__builtin_expect(__any_sync(~0u, grow), 0)) {
                        const float f = grow ? exp2_fast(m - top) : 1.0f;
                        m = grow ? top : m;
                        l *= f;
#pragma unroll
                        for (int c = 0; c < DP / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(oc + 32 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(oc + 32 * c, o);
                        }
                    }
                }
                const float2 mul2 = make_float2(mul, mul), neg = make_float2(-m, -m);
                float2 sum[4] = {};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float2 x = __ffma2_rn(make_float2(s[64 * c + 2 * e], s[64 * c + 2 * e + 1]), mul2, neg);
                        x.x = exp2_fast(x.x);
                        x.y = exp2_fast(x.y);
                        sum[e & 3] = __fadd2_rn(sum[e & 3], x);
                        p[e] = pack_bf16x2(x.x, x.y); // an operand of the second product: bf16, as v is
                    }
                    tmem_st32(sc + 32 * c, p);
                }
                sum[0] = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
                l += sum[0].x + sum[0].y;
                if (__builtin_expect(r == 0 && valid < kTile && w.kend < a.Nk, 0)) { // v rows behind the length
                    const uint32_t pos = it + 2 * j + 1, vs = pos % NST;
                    if (!wait_or_abort(smem_addr(&kvfull[vs]), (pos / NST) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    unsigned char *v = smem_raw + (kvbase + vs * TB - smem_addr(smem_raw));
                    const int tid = threadIdx.x;
                    for (int e = valid * 8 + tid; e < kTile * 8; e += 128)
#pragma unroll
                        for (int sub = 0; sub < NSUB; ++sub)
                            *reinterpret_cast<uint4 *>(v + sub * SUB + e * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&pfull[r]));
                __syncwarp(); // the arrival goes out before any lane begins to wait
            }
            if (!ok)
                break;
            if (w.ntiles > 0) {
                if (!wait_or_abort(smem_addr(&ofull[r]), nitem & 1u, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                ++nitem;
                it += 2 * w.ntiles;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l; // (a sum of NaN gives NaN, no key 0)
            if (__builtin_expect(w.part < 0, 1)) {
                uint32_t o[DP] = {};
                if (w.ntiles > 0) {
#pragma unroll
                    for (int c = 0; c < NSUB; ++c)
                        tmem_ld64(oc + 64 * c, reinterpret_cast<uint32_t(&)[64]>(o[64 * c]));
                    tmem_wait_ld();
                }
                __nv_bfloat16 *dst = a.o.row(w.b, iq, h);
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    uint32_t v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = pack_bf16x2(__uint_as_float(o[16 * c + 2 * k]) * inv,
                                           __uint_as_float(o[16 * c + 2 * k + 1]) * inv);
                    if (live)
                        store16(dst + 16 * c, v, a.D - 16 * c, t.wide);
                }
            } else if (w.ntiles > 0) { // (a split without keys has m = -inf: its o is not read)
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(oc + 32 * c, o);
                    tmem_wait_ld();
                    float *dst = a.part + part_row(t, w, row) * a.D + 32 * c;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (live && 32 * c + 8 * e < a.D)
                            Row<float, 8, true>::store(dst + 8 * e, reinterpret_cast<const float *>(o) + 8 * e);
                }
            }
            tc_fence_before();
            if (live) {
                if (w.part < 0) {
                    if (a.lse)
                        a.lse[stat] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                } else {
                    part_stats(t)[part_row(t, w, row)] = make_float2(w.ntiles > 0 ? m : -INFINITY, l);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort)
        atomicAdd(&g_attn_timeouts, 1u);
}

// One warp per query row of a split item.
__global__ void __launch_bounds__(128) attn_tail_join_kernel(const TcArgs t)
{
    asm volatile("griddepcontrol.wait;" ::: "memory"); // the grid before has written its parts
    const AttnArgs &a = t.a;
    const int64_t rows = (int64_t)t.tail * (2 * kTile), at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    Item w;
    place(t, t.whole + (int)(at / (2 * kTile)), w);
    const int row = w.row0 + (int)(at % (2 * kTile)), iq = row >> t.lgp, h = w.hs * t.gp + (row & (t.gp - 1));
    if (iq >= a.Nq)
        return;
    join_parts(a.part + at * a.D, part_stats(t) + at, rows, a.splits, a.D, a.o.row(w.b, iq, h), a.lse ? a.lse + ((int64_t)w.b * a.Hq + h) * a.Nq + iq : nullptr);
}

// Items of 256 query rows, the last round's split over the keys.  (2 x 3520 x 3520, 16 heads: 448 items,
// 4 of them shared: 186 us, 225 without.)
Rounds plan(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D)
{
    const int64_t gp = attn_tc_group((int)(Hq / Hkv));
    return Rounds(B * (Hq / gp) * ((Nq * gp + 2 * kTile - 1) / (2 * kTile)), (Nk + kTile - 1) / kTile, kMaxSplits,
                  D > 64 ? 2.0 : 1.75, 3, 2.0 * 2 * kTile * 4 * D / 6.0e6);
}

template <int DP> tok_status launch(const TcArgs &t, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                                    cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(attn_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes<DP>());
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    const int sms = sm_count();
    attn_fwd_kernel<DP><<<std::min(t.items, sms > 0 ? sms : 1), kThreads, smem_bytes<DP>(), stream>>>(q, k, v, t);
    const tok_status st = launch_status();
    return st == TOK_OK && t.tail > 0 ? launch_join(attn_tail_join_kernel, (int64_t)t.tail * (2 * kTile), t, stream) : st;
}

} // namespace

int64_t attn_tc_workspace(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D)
{
    const Rounds r = plan(B, Nq, Nk, Hq, Hkv, D);
    return r.tail * r.shares * 2 * kTile * (D + 2) * 4;
}

// Heads that a 128-row tile holds: the group, where it divides the tile.
int attn_tc_group(int G) { return G <= kTile && (G & (G - 1)) == 0 ? G : 1; }

tok_status attn_tc_forward(const AttnArgs &a, cudaStream_t stream)
{
    TcArgs t{};
    t.a = a;
    t.gp = attn_tc_group(a.G);
    while (t.gp >> t.lgp > 1)
        ++t.lgp;
    t.wide = rows_wide(a.o, a.B, a.Nq, a.Hq);
    t.hsets = a.Hq / t.gp;
    t.nqt = (int)(((int64_t)a.Nq * t.gp + 2 * kTile - 1) / (2 * kTile));
    t.nqt_div = FastDiv((uint32_t)t.nqt);
    t.hsets_div = FastDiv((uint32_t)t.hsets);
    const Rounds r = plan(a.B, a.Nq, a.Nk, a.Hq, a.Hkv, a.D);
    t.a.splits = (int)r.shares;
    t.whole = (int)r.whole;
    t.tail = (int)r.tail;
    t.items = (int)(r.whole + r.tail * r.shares);
    t.qb = a.B > 1 && a.q.b == 0 ? 0 : 1;
    t.kb = a.B > 1 && a.k.b == 0 ? 0 : 1;
    t.vb = a.B > 1 && a.v.b == 0 ? 0 : 1;
    t.kh = a.Hkv > 1 && a.k.h == 0 ? 0 : 1;
    t.vh = a.Hkv > 1 && a.v.h == 0 ? 0 : 1;
    CUtensorMap q, k, v;
    if (!heads_map(&q, a.q, a.B, a.Nq, a.Hq, a.D, t.gp, kTile / t.gp) ||
        !heads_map(&k, a.k, a.B, a.Nk, a.Hkv, a.D, 1, kTile) || !heads_map(&v, a.v, a.B, a.Nk, a.Hkv, a.D, 1, kTile))
        return TOK_ERR_SHAPE;
    return a.D <= 64 ? launch<64>(t, q, k, v, stream) : launch<128>(t, q, k, v, stream);
}

tok_status read_and_clear_attn_timeouts(cudaStream_t stream, unsigned int *count)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_attn_timeouts, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost,
                                              stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && *count)
        e = cudaMemcpyToSymbolAsync(g_attn_timeouts, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    return TOK_OK;
}

} // namespace tok
