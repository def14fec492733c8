// Attention of a few new tokens of each stream over its keys and values in pages.
//
// The call is bound by reading the keys and values once.  16 query rows (queries x the heads of a group) of one key
// head are a unit; its keys come in rounds of 64, 16 to each of a CTA's 4 warps, on warp-level m16n8k16 tiles with a running maximum
// and sum per warp.  Streams differ in length, so the rounds of all units of all streams, in order, are one sequence,
// which two CTAs per SM share out in equal contiguous parts.  A CTA that has a unit whole writes its
// result; of a unit that several CTAs have parts of, partial results (fp32) go to the workspace, at most two per CTA,
// and join_kernel, launched early, adds them up in order.
//
// Each warp keeps a ring of its own in shared memory, all stages but one on their way (cp.async, 16 bytes a lane, so
// that pages of any size and stride are read whole rows at a time); the ring runs on from one unit
// into the next.  A table entry is loaded one step before its rows.
#include <algorithm>

#include "pages.cuh"

namespace tok {
namespace {

constexpr int kRows = 16; // query rows of a unit
constexpr int kWarps = 4;
constexpr int kStep = 16;               // keys of a warp's step
constexpr int kRound = kWarps * kStep;  // keys of a CTA's
constexpr int kMinRounds = 2;           // fewest rounds of a CTA
constexpr int kCtas = 148 * 2;
constexpr int64_t kMaxNq = 64;

struct PagedArgs {
    HeadsView q, o;
    PagesView k, v;
    const int32_t *table, *k_lens, *q_lens;
    float *lse;
    float *part;   // [kCtas][2][kRows][D]: unit begun before the CTA's part, unit going on behind it
    float2 *stats; // [kCtas][2][kRows]: their maximum and sum
    int2 *spans;   // [units]: first and last CTA of a unit, or (-1, .) of one that a CTA has whole
    int64_t table_row;
    int B, Nq, Hq, Hkv, G, D, tiles, units, P, tokens; // row tiles; units of a stream; tokens of a table row
    FastDiv page;
    float scale2;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) // zeros where !ok
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// NP = ceil(D / 64).  Row r of a tile of 16 keeps its 16-byte chunk c at c ^ mix(r): the 8 lanes that a shared-memory
// read serves at a time (key fragments: 2 rows x 4 chunks; value fragments: 4 rows of one parity x 2 chunks) then meet 8
// different banks.
template <int NP> struct Ring {
    static constexpr int stages = NP == 2 ? 3 : 4;
    static constexpr int row = NP * 128, tile = kStep * row, stage = 2 * tile, warp = stages * stage; // bytes
    static constexpr int join = 32 * NP * 32 * 4; // a warp's result
    static constexpr int bytes = kWarps * warp + 2 * join;
};
__device__ __forceinline__ int mix(int r) { return (r & 6) ^ ((r & 1) << 2); }

__device__ __forceinline__ int rounds_of(const PagedArgs &a, int b, int &len)
{
    len = min(max(a.k_lens[b], 0), a.tokens);
    return max(1, (len + kRound - 1) / kRound); // (a stream without keys has its rows written in one round)
}

__device__ __forceinline__ int query_count(const PagedArgs &a, int b)
{
    return a.q_lens ? min(max(a.q_lens[b], 0), a.Nq) : a.Nq;
}

// Keys that a row of a unit sees.
__device__ __forceinline__ int limit_of(const PagedArgs &a, int row, int len, int queries)
{
    const int i = row / a.G;
    return row < a.Nq * a.G && i < queries ? min(max(len - queries + i + 1, 0), len) : 0;
}

// A place in the sequence of rounds.
struct Place {
    int b, unit, round, rounds, len;
};

template <int NP>
__global__ void __launch_bounds__(kWarps * 32, 2) paged_kernel(const PagedArgs a)
{
    constexpr int NC = 2 * NP;
    using R = Ring<NP>;
    extern __shared__ __align__(128) unsigned char ring_raw[];
    __shared__ float sm[kWarps][kRows], sl[kWarps][kRows];
    __shared__ int64_t s_sum[kWarps];
    __shared__ Place s_first;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- This CTA's part [pos, end) of the rounds. ----
    auto block_sum = [&](int64_t v, int64_t &before) { // sum over the block; `before`: of the threads before
        int64_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(~0u, x, o);
            if (lane >= o)
                x += y;
        }
        __syncthreads();
        if (lane == 31)
            s_sum[warp] = x;
        __syncthreads();
        before = x - v;
        int64_t all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? s_sum[w] : 0;
            all += s_sum[w];
        }
        return all;
    };
    int64_t total = 0, before;
    for (int b0 = 0; b0 < a.B; b0 += kWarps * 32) {
        int len;
        total += block_sum(b0 + tid < a.B ? (int64_t)rounds_of(a, b0 + tid, len) * a.units : 0, before);
    }
    const int64_t ctas = min((int64_t)kCtas, max((int64_t)1, total / kMinRounds)), cta = blockIdx.x;
    if (cta >= ctas)
        return;
    int64_t pos = total * cta / ctas;
    const int64_t end = total * (cta + 1) / ctas;
    int64_t run = 0;
    for (int b0 = 0; b0 < a.B; b0 += kWarps * 32) {
        const int b = b0 + tid;
        int len = 0;
        const int rounds = b < a.B ? rounds_of(a, b, len) : 0;
        const int64_t mine = (int64_t)rounds * a.units, all = block_sum(mine, before), at = run + before;
        if (pos >= at && pos < at + mine) {
            const int64_t in = pos - at;
            s_first = Place{b, (int)(in / rounds), (int)(in % rounds), rounds, len};
        }
        run += all;
        if (run > pos)
            break;
    }
    __syncthreads();
    Place now = s_first, ahead = now;
    auto advance = [&](Place &p) {
        if (++p.round < p.rounds)
            return;
        p.round = 0;
        if (++p.unit < a.units)
            return;
        p.unit = 0;
        if (++p.b < a.B)
            p.rounds = rounds_of(a, p.b, p.len);
    };

    // ---- Copies: `ahead` is the round whose table entry is at hand. ----
    unsigned char *ring = ring_raw + warp * R::warp;
    const uint32_t ring_s = smem_addr(ring);
    constexpr int kChunks = NP * 8, kCopies = kStep * kChunks / 32; // per tile and lane
    int entry = -1, in_page = 0; // lane r (and r + 16): of key r of the step; -1: there is none, -2: not a page
    auto look_up = [&]() {
        const int key = ahead.round * kRound + warp * kStep + (lane & 15);
        entry = -1;
        if (key < ahead.len) {
            const uint32_t p = a.page.div((uint32_t)key);
            in_page = (int)(key - p * a.page.d);
            entry = a.table[ahead.b * a.table_row + p];
        }
    };
    int64_t left = end - pos; // rounds not yet fetched
    uint32_t bad = 0;         // stages with a key of no page
    auto fetch = [&](int stage) {
        if (left > 0) {
            const bool none = entry == -1 && ahead.round * kRound + warp * kStep + (lane & 15) >= ahead.len;
            const bool out = !none && (uint32_t)entry >= (uint32_t)a.P;
            if (__any_sync(~0u, out))
                bad |= 1u << stage;
            const int page = none || out ? -1 : entry;
            const int64_t head = ahead.unit / a.tiles;
            const __nv_bfloat16 *kbase = a.k.p + head * a.k.h, *vbase = a.v.p + head * a.v.h;
            const uint32_t dst = ring_s + stage * R::stage;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int e = i * 32 + lane, r = e / kChunks, ch = e % kChunks;
                const int pg = __shfl_sync(~0u, page, r), in = __shfl_sync(~0u, in_page, r);
                const bool ok = pg >= 0 && ch * 8 < a.D;
                const uint32_t to = dst + r * R::row + ((ch ^ mix(r)) << 4);
                copy16(to, ok ? kbase + (pg * a.k.pg + in * a.k.t + ch * 8) : a.q.p, ok);
                copy16(to + R::tile, ok ? vbase + (pg * a.v.pg + in * a.v.t + ch * 8) : a.q.p, ok);
            }
            if (--left > 0) {
                advance(ahead);
                look_up();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up();
#pragma unroll
    for (int s = 0; s < R::stages - 1; ++s)
        fetch(s);

    // ---- Rounds. ----
    uint4 qlo[NC], qhi[NC];
    float acc[NP][8][4];
    float mlo, mhi, llo, lhi;
    int lim_lo = 0, lim_hi = 0, lim_first = 0; // keys seen by this lane's rows; by all of the unit's
    bool unit_bad = false, whole = false;
    int stage = 0;
    bool fresh = true;
    for (; pos < end; ++pos) {
        const int hk = now.unit / a.tiles, r0 = (now.unit - hk * a.tiles) * kRows;
        if (fresh) {
            fresh = false;
            whole = now.round == 0;
            const int queries = query_count(a, now.b), lo = r0 + g, hi = lo + 8, rows = a.Nq * a.G;
            lim_lo = limit_of(a, lo, now.len, queries);
            lim_hi = limit_of(a, hi, now.len, queries);
            lim_first = limit_of(a, r0, now.len, queries);
            load_chan<NC>(qlo, a.q.row(now.b, lo / a.G, hk * a.G + lo % a.G), lo < rows, 8 * c, a.D);
            load_chan<NC>(qhi, a.q.row(now.b, hi / a.G, hk * a.G + hi % a.G), hi < rows, 8 * c, a.D);
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[p][j][e] = 0.0f;
            mlo = mhi = -INFINITY;
            llo = lhi = 0.0f;
            unit_bad = false;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(R::stages - 2) : "memory"); // this lane's copies of the round
        __syncwarp(); // every lane's; and every lane is done with the stage refilled next
        const int kk = now.round * kRound + warp * kStep;
        unit_bad = unit_bad || (bad >> stage & 1);
        bad &= ~(1u << stage);
        fetch(stage == 0 ? R::stages - 1 : stage - 1);
        const unsigned char *kt = ring + stage * R::stage, *vt = kt + R::tile;
        stage = stage + 1 == R::stages ? 0 : stage + 1;
        if (kk < now.len) {
            float s[2][4] = {};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint4 kf[NC];
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    kf[i] = *reinterpret_cast<const uint4 *>(kt + (8 * t + g) * R::row + (((4 * i + c) ^ mix(g)) << 4));
                mma_chan<NC>(s[t], qlo, qhi, kf);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[t][e] = kk + 8 * t + 2 * c + (e & 1) < (e < 2 ? lim_lo : lim_hi) ? s[t][e] * a.scale2 : -INFINITY;
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
            // A value that some rows see and others do not meets weights of 0; where it is no finite
            // number, the products are taken key by key, with the rows that see the key.
            bool careful = false;
            if (kk + kStep > lim_first) {
                uint32_t odd = 0;
#pragma unroll
                for (int i = 0; i < kStep * kChunks / 32; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(vt + (i * 32 + lane) * 16);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        odd |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
                }
                careful = __any_sync(~0u, odd);
            }
            if (!careful) {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    RowFrag vf;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 2 * c + (i & 1) + 8 * (i >> 1);
                        vf.r[i] = *reinterpret_cast<const uint4 *>(vt + r * R::row + (((8 * p + g) ^ mix(r & 7)) << 4));
                    }
                    mma_rows(acc[p], pa, vf);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < kStep; ++k) { // key k's weights are in lane k % 8 / 2 of a row's four
                    const int from = (lane & ~3) | (k & 7) >> 1;
                    const uint32_t plo = __shfl_sync(~0u, k < 8 ? pa[0] : pa[2], from);
                    const uint32_t phi = __shfl_sync(~0u, k < 8 ? pa[1] : pa[3], from);
                    const float wlo = k & 1 ? bf16_hi(plo) : bf16_lo(plo), whi = k & 1 ? bf16_hi(phi) : bf16_lo(phi);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        float x[2][8];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            Row<__nv_bfloat16, 8, true>::load(
                                reinterpret_cast<const __nv_bfloat16 *>(vt + k * R::row + (((8 * p + 2 * c + h) ^ mix(k & 7)) << 4)),
                                x[h]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (kk + k < lim_lo) {
                                acc[p][j][0] += wlo * x[0][j];
                                acc[p][j][1] += wlo * x[1][j];
                            }
                            if (kk + k < lim_hi) {
                                acc[p][j][2] += whi * x[0][j];
                                acc[p][j][3] += whi * x[1][j];
                            }
                        }
                    }
                }
            }
        }
        const bool done = now.round + 1 == now.rounds;
        if (!done && pos + 1 < end) {
            ++now.round;
            continue;
        }

        // ---- The unit's end, or that of this CTA's part: the warps' results added up. ----
        fresh = true;
        llo = quad_sum(llo); // (all lanes, whatever their rows see)
        lhi = quad_sum(lhi);
        llo = lim_lo == 0 ? 0.0f : unit_bad ? __int_as_float(0x7FC00000) : llo;
        lhi = lim_hi == 0 ? 0.0f : unit_bad ? __int_as_float(0x7FC00000) : lhi;
        if (c == 0) {
            sm[warp][g] = mlo;
            sm[warp][g + 8] = mhi;
            sl[warp][g] = llo;
            sl[warp][g + 8] = lhi;
        }
        __syncthreads();
        float all_lo = sm[0][g], all_hi = sm[0][g + 8];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            all_lo = fmaxf(all_lo, sm[w][g]);
            all_hi = fmaxf(all_hi, sm[w][g + 8]);
        }
        llo = lhi = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            llo += (sm[w][g] == -INFINITY ? 0.0f : exp2_fast(sm[w][g] - all_lo)) * sl[w][g];
            lhi += (sm[w][g + 8] == -INFINITY ? 0.0f : exp2_fast(sm[w][g + 8] - all_hi)) * sl[w][g + 8];
        }
        const float flo = mlo == -INFINITY ? 0.0f : exp2_fast(mlo - all_lo);
        const float fhi = mhi == -INFINITY ? 0.0f : exp2_fast(mhi - all_hi);
        float4 *buf = reinterpret_cast<float4 *>(ring_raw + kWarps * R::warp);
        constexpr int kBuf = R::join / 16;
        auto give = [&](float4 *to) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    to[(p * 8 + j) * 32 + lane] = make_float4(acc[p][j][0], acc[p][j][1], acc[p][j][2], acc[p][j][3]);
        };
        auto take = [&](const float4 *from) {
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 x = from[(p * 8 + j) * 32 + lane];
                    acc[p][j][0] += x.x;
                    acc[p][j][1] += x.y;
                    acc[p][j][2] += x.z;
                    acc[p][j][3] += x.w;
                }
        };
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[p][j][0] *= flo;
                acc[p][j][1] *= flo;
                acc[p][j][2] *= fhi;
                acc[p][j][3] *= fhi;
            }
        if (warp & 1)
            give(buf + (warp >> 1) * kBuf);
        __syncthreads();
        if (!(warp & 1))
            take(buf + (warp >> 1) * kBuf);
        __syncthreads();
        if (warp == 2)
            give(buf);
        __syncthreads();
        if (warp == 0) {
            take(buf);
            const bool alone = whole && done;
            const int64_t unit = (int64_t)now.b * a.units + now.unit;
            if (lane == 0 && whole) {
                const int64_t last = pos + (now.rounds - 1 - now.round); // (round 0 was at pos - now.round)
                a.spans[unit] = alone ? make_int2(-1, -1) : make_int2((int)cta, (int)(((last + 1) * ctas - 1) / total));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = r0 + g + 8 * h;
                if (row >= a.Nq * a.G)
                    continue;
                const float m = h ? all_hi : all_lo, l = h ? lhi : llo;
                const int iq = row / a.G, head = hk * a.G + row % a.G;
                if (alone) {
                    const float inv = 1.0f / l;
                    __nv_bfloat16 *o = a.o.row(now.b, iq, head);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                x[j] = l == 0.0f ? 0.0f : acc[p][j][2 * h + e] * inv;
                            const int d = 64 * p + 16 * c + 8 * e;
                            if (d < a.D)
                                Row<__nv_bfloat16, 8, true>::store(o + d, x);
                        }
                    if (c == 0 && a.lse)
                        a.lse[((int64_t)now.b * a.Hq + head) * a.Nq + iq] =
                            l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                } else {
                    const int64_t at = (cta * 2 + whole) * kRows + (row - r0);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float x[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                x[j] = acc[p][j][2 * h + e];
                            const int d = 64 * p + 16 * c + 8 * e;
                            if (d < a.D)
                                Row<float, 8, true>::store(a.part + at * a.D + d, x);
                        }
                    if (c == 0)
                        a.stats[at] = make_float2(m, l);
                }
            }
        }
        advance(now);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// One warp per query row and head: the parts of its unit in order.
__global__ void __launch_bounds__(128) paged_join_kernel(const PagedArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory"); // the grid before has written its parts
    const int lane = threadIdx.x & 31;
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); // (b, query, head)
    if (at >= (int64_t)a.B * a.Nq * a.Hq)
        return;
    const int64_t bq = at / a.Hq;
    const int head = (int)(at - bq * a.Hq), b = (int)(bq / a.Nq), iq = (int)(bq - (int64_t)b * a.Nq);
    const int hk = head / a.G, row = iq * a.G + head % a.G;
    const int2 span = a.spans[(int64_t)b * a.units + hk * a.tiles + row / kRows];
    if (span.x < 0)
        return;
    const int n = span.y - span.x + 1, r = row % kRows;
    auto place = [&](int i) { return ((int64_t)(span.x + i) * 2 + (i == 0)) * kRows + r; }; // (the first begins it)
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32)
        m = fmaxf(m, a.stats[place(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    float l = 0.0f, v[4] = {};
    const int d = 4 * lane;
    for (int i0 = 0; i0 < n; i0 += 32) {
        float f = 0.0f;
        if (i0 + lane < n) {
            const float2 x = a.stats[place(i0 + lane)];
            f = x.x == -INFINITY ? 0.0f : exp2_fast(x.x - m);
            l += f * x.y; // (0 times NaN: a part whose scores were no numbers)
            f = x.y != x.y ? x.y : f;
        }
        const int n1 = min(32, n - i0);
#pragma unroll 8
        for (int i = 0; i < n1; ++i) {
            const float fi = __shfl_sync(~0u, f, i);
            if (d < a.D && fi != 0.0f) {
                float x[4];
                Row<float, 4, true>::load(a.part + place(i0 + i) * a.D + d, x);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] += fi * x[j];
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        l += __shfl_xor_sync(~0u, l, o);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (d < a.D) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] *= inv;
        Row<__nv_bfloat16, 4, true>::store(a.o.row(b, iq, head) + d, v);
    }
    if (lane == 0 && a.lse)
        a.lse[((int64_t)b * a.Hq + head) * a.Nq + iq] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

struct PagedDims {
    int64_t B, Nq, Hq, Hkv, D;
    bool ok() const
    {
        int64_t p;
        return B >= 0 && B <= 65535 && Nq >= 0 && Nq <= kMaxNq && Hkv >= 1 && Hq >= 1 && Hq <= 65535 && Hq % Hkv == 0 &&
               D >= 8 && D <= 128 && D % 8 == 0 && prod_ok({B, Hq, Nq}, &p) && p < ((int64_t)1 << 30);
    }
    int64_t tiles() const { return (Nq * (Hq / Hkv) + kRows - 1) / kRows; }
    int64_t units() const { return Hkv * tiles(); } // of a stream
    int64_t at_stats() const { return (int64_t)kCtas * 2 * kRows * D * 4; }
    int64_t at_spans() const { return at_stats() + (int64_t)kCtas * 2 * kRows * 8; }
    int64_t workspace() const { return B == 0 || Nq == 0 ? 0 : at_spans() + B * units() * 8; }
};

template <int NP> tok_status launch(const PagedArgs &a, cudaStream_t stream)
{
    const cudaError_t e =
        cudaFuncSetAttribute(paged_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<NP>::bytes);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    paged_kernel<NP><<<kCtas, kWarps * 32, Ring<NP>::bytes, stream>>>(a);
    const tok_status st = launch_status();
    return st == TOK_OK ? launch_join(paged_join_kernel, (int64_t)a.B * a.Nq * a.Hq, a, stream) : st;
}

constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;

} // namespace
} // namespace tok

extern "C" int64_t tok_paged_attention_workspace_size(int64_t B, int64_t Nq, int64_t Hq, int64_t Hkv, int64_t D)
{
    const tok::PagedDims d{B, Nq, Hq, Hkv, D};
    return d.ok() ? d.workspace() : -1;
}

extern "C" tok_status tok_paged_attention(const tok_heads *q, const tok_pages *k_pages, const tok_pages *v_pages,
                                          const int32_t *table, const int32_t *k_lens, const int32_t *q_lens,
                                          const tok_heads *o, float *lse, int64_t B, int64_t Nq, int64_t Hq,
                                          int64_t Hkv, int64_t D, int64_t P, int64_t page_size, int64_t M,
                                          int64_t table_row, float scale, void *workspace, int64_t workspace_bytes,
                                          cudaStream_t stream)
{
    using namespace tok;
    const PagedDims dim{B, Nq, Hq, Hkv, D};
    int64_t slots, tokens;
    if (!dim.ok() || P < 0 || M < 0 || page_size < 1 || page_size > kIntMax || !prod_ok({P, page_size}, &slots) ||
        slots > kIntMax || !prod_ok({M, page_size}, &tokens) || tokens > kIntMax - kRound)
        return TOK_ERR_SHAPE;
    if (B == 0 || Nq == 0)
        return TOK_OK;
    if (B > 1 && (table_row < M || table_row >= ((int64_t)1 << 38) / B))
        return TOK_ERR_SHAPE;
    if (!q || !k_pages || !v_pages || !o || !q->ptr || !o->ptr || !k_lens || (M > 0 && !table) ||
        (P > 0 && (!k_pages->ptr || !v_pages->ptr)))
        return TOK_ERR_NULL;
    const View vq{q, B, Nq, Hq, D, false}, vo{o, B, Nq, Hq, D, false};
    const PoolView pk{k_pages, P, page_size, Hkv, D}, pv{v_pages, P, page_size, Hkv, D};
    if (!vq.strides_ok() || !vo.strides_ok() || !pk.strides_ok() || !pv.strides_ok() || !vo.distinct())
        return TOK_ERR_SHAPE;
    const int64_t need = dim.workspace();
    if (workspace_bytes < need)
        return TOK_ERR_SHAPE;
    if (!workspace)
        return TOK_ERR_NULL;
    if (!vq.aligned16() || !vo.aligned16() || (P > 0 && (!pk.aligned16() || !pv.aligned16())) || !aligned(table, 4) ||
        !aligned(k_lens, 4) || !aligned(q_lens, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
        return TOK_ERR_ALIGN;
    const int64_t stats = B * Hq * Nq * 4, tb = 4 * ((B - 1) * table_row + M);
    struct Out {
        const void *p;
        int64_t bytes;
    };
    if (meet(vo, vq))
        return TOK_ERR_ALIAS;
    for (const Out &w : {Out{lse, stats}, Out{workspace, need}})
        if (w.p && (meets(vq, w.p, w.bytes) || meets(vo, w.p, w.bytes)))
            return TOK_ERR_ALIAS;
    for (const Out &w : {Out{o->ptr, vo.span() * 2}, Out{lse, stats}, Out{workspace, need}})
        if (w.p && (overlaps(w.p, w.bytes, k_lens, 4 * B) || (q_lens && overlaps(w.p, w.bytes, q_lens, 4 * B)) ||
                    (M > 0 && overlaps(w.p, w.bytes, table, tb)) ||
                    (P > 0 && (pk.meets(w.p, w.bytes) || pv.meets(w.p, w.bytes)))))
            return TOK_ERR_ALIAS;
    if (lse && overlaps(lse, stats, workspace, need))
        return TOK_ERR_ALIAS;

    PagedArgs a{};
    a.q = view(q);
    a.o = view(o);
    a.k = view(k_pages);
    a.v = view(v_pages);
    a.table = table;
    a.k_lens = k_lens;
    a.q_lens = q_lens;
    a.lse = lse;
    char *ws = static_cast<char *>(workspace);
    a.part = reinterpret_cast<float *>(ws);
    a.stats = reinterpret_cast<float2 *>(ws + dim.at_stats());
    a.spans = reinterpret_cast<int2 *>(ws + dim.at_spans());
    a.table_row = table_row;
    a.B = (int)B;
    a.Nq = (int)Nq;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.D = (int)D;
    a.tiles = (int)dim.tiles();
    a.units = (int)dim.units();
    a.P = (int)P;
    a.tokens = (int)tokens;
    a.page = FastDiv((uint32_t)page_size);
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    return D <= 64 ? launch<1>(a, stream) : launch<2>(a, stream);
}
