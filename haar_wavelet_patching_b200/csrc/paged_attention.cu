// Attention of a few new tokens of each stream over its keys and values in pages.
//
// The call is bound by reading the keys and values once.  Up to 64 query rows (queries x the heads of a group) of one
// key head are a unit; its keys come in rounds of 128.  Streams differ in length, so the rounds of all units of all
// streams, in order, are one sequence, which the SMs' CTAs share out in equal contiguous parts.  A CTA that has a
// unit whole writes its result; of a unit that several CTAs have parts of, partial results (fp32) go to the
// workspace, at most two per CTA, and paged_join_kernel, launched early, adds them up in order.
//
// There are few query rows and many keys, so the products are taken transposed, with the 128 rows of the tensor
// cores' tiles for keys and for channels: scores^T = K Q^T (128 keys x N queries), then o^T += V^T P^T
// (channels x 2 N, the weights and what their rounding has left; one column more or less is no time), and no thread
// touches a key or a value.  A CTA's warps:
//   warps 0-3  softmax, a key to a thread (its lane of tensor memory): scores -> weights, a bf16 number and another
//              for the rest of each, into shared memory as the second product's operand.  Weights are relative to the
//              score of the unit's first key, and to the largest one from where one exceeds it by more than 2^16
//              (every term carries the same factor, so the quotient is unchanged); a vote of the four warps each
//              round says so.  Sums stay with the threads up to a unit's end: o / sum -> HBM;
//   warps 4, 7 tensor copies of keys and of values into rings of 128-byte-swizzled tiles: boxes of as many rows as
//              divide both a page and a round, or four rows of any places;
//   warp 5     one thread issues the MMAs: the next round's scores before this round's second product;
//   warp 6     copies of the units' queries and what their rows are, one unit ahead.
// A round may read rows behind a stream's last token: their scores are masked and their values zeroed in shared memory.
// All waits are bounded as in the convolutions.
//
// Measured, bf16: 4 streams x 56,320 keys, 8 key heads x 128: 146 us (923 MB, 6.3 TB/s); 16 streams of up to 3520
// keys, in pages of 16, 31 us (floor 18.8), of which about 6 are the launch, the shares and the first copies, and 5
// the join; drafts of 5 to a stream on pages of 24: 22.5 us, the same chain.
// With more than 32 rows of a key head the softmax warps' instructions bound it (64 rows of a key to a thread):
// 4 x 56,320 keys, 36 rows, 128 channels 326 us (298 with weights rounded once, which are off by up to 2^-9),
// 64 channels 302 (268).
#include <algorithm>
#include <numeric>

#include "pages.cuh"

namespace tok {

static __device__ unsigned int g_paged_timeouts = 0;

namespace {

constexpr int kRound = 128;    // keys of a round
// A unit's beginning and end take a CTA about as long as this many rounds; fewest places of a CTA.
constexpr int kEnd = 1, kMinPlaces = 4;
constexpr int kCtas = 148;
constexpr int64_t kMaxNq = 64;
constexpr int kThreads = 8 * 32;
constexpr float kGrow = 16.0f; // log2 of the largest weight
constexpr float kLowest = -3.402823466e+38f;

struct PagedArgs {
    HeadsView q, o;
    PagesView k, v;
    const int32_t *table, *k_lens, *q_lens;
    float *lse;
    float *part;   // [kCtas][2][rows][D]: unit begun before the CTA's part, unit going on behind it
    float2 *stats; // [kCtas][2][rows]: their maximum and sum
    float *side;   // [kCtas][64][rows]: scores of keys whose values are no numbers
    int2 *spans;   // [units]: first and last CTA of a unit, or (-1, .) of one that a CTA has whole
    int64_t table_row;
    int B, Nq, Hq, Hkv, G, D;
    int rows, tiles, units, P, tokens; // rows of a unit; row tiles; units of a stream; pages; tokens of a table row
    FastDiv page, group;
    int none;         // the page of copies that bring zeros (PoolMap)
    int box_rows;     // rows of a tensor copy
    int kh, vh;       // coordinate factors: 0 for broadcast heads
    // Small boxes: rows of any places, four to a copy, of a map in which page, token and head are one coordinate.
    struct Gather {
        int page, token, head, rows; // what one of each adds; the map's rows (0: not so)
    } gk, gv;
    float scale2;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) // zeros where !ok
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}

// Barrier of the softmax warps; `any`: whether one of their threads says so.
__device__ __forceinline__ void softmax_sync()
{
    __syncwarp();
    asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool softmax_any(bool v)
{
    uint32_t r;
    __syncwarp();
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)v)
                 : "memory");
    return r != 0;
}

// One value of each of 16 rows per lane -> the rows' maxima (or sums) over the warp: lane 2 i has row i's.
template <bool kMax> __device__ __forceinline__ float reduce16(float (&v)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 8; o; o >>= 1) { // o rows left of 2 o: the upper ones go to the lane with bit 2 o set
        const bool up = lane & (2 * o);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < o) {
                const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
                const float x = __shfl_xor_sync(~0u, give, 2 * o);
                v[i] = kMax ? fmaxf(keep, x) : keep + x;
            }
    }
    const float x = __shfl_xor_sync(~0u, v[0], 1);
    return kMax ? fmaxf(v[0], x) : v[0] + x;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15}, [%16];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                   "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16};" ::"r"(taddr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]),
                 "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
                 : "memory");
}

// Tensor copy of data that is read once: first to leave L2, so that code, tables and partial results stay there.
__device__ __forceinline__ void tma_load_4d_once(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                                 uint32_t bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
                 "[%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
                 "l"((uint64_t)map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void tma_gather4_once(uint32_t dst, const CUtensorMap *map, int x, const int (&y)[4], uint32_t bar,
                                                 uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
                 "[%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
                 "l"((uint64_t)map), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ uint64_t evict_first()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

constexpr uint32_t kATransposed = 1u << 15; // instruction descriptor: A is MN-major

__device__ __forceinline__ int rounds_of(const PagedArgs &a, int b, int &len)
{
    len = min(max(a.k_lens[b], 0), a.tokens);
    return max(1, (len + kRound - 1) / kRound); // (a stream without keys has its rows written in one round)
}

__device__ __forceinline__ int query_count(const PagedArgs &a, int b)
{
    return a.q_lens ? min(max(a.q_lens[b], 0), a.Nq) : a.Nq;
}

// A place in the sequence of rounds.
struct Place {
    int b, unit, round, rounds, len;
};

// Shared memory of a CTA: DP channels, N query rows; `ring` rounds of keys and values.
template <int DP, int N> struct Smem {
    static constexpr int sub = kRound * 128;     // 64 channels of a round's keys
    static constexpr int tile = DP / 64 * sub;   // keys or values of a round
    static constexpr int q = DP / 64 * N * 128;  // a unit's queries
    // Columns of the second product: the weights rounded to bf16, as the values are, and behind them what that has
    // left, so that the output's rounding alone counts.  A key's are a line of shared memory; with 64 rows they are
    // two, as a line of the swizzle has 128 bytes, in tiles of their own: first the weights' two (of rounds in turn),
    // then the rests', of which there is one where the room is short: it is written once the product before has read
    // it.
    static constexpr int wide = 2 * N;
    static constexpr bool split = N == 64;
    static constexpr int line = split ? 2 * N : 2 * wide, p = kRound * line; // a round's weights
    static constexpr int rests = !split ? 0 : DP == 64 ? 2 : 1;
    static constexpr int units = N == 64 ? 2 : N == 16 && DP == 128 ? 3 : 4; // whose queries may be there
    static constexpr int ring = DP == 64 ? (N == 16 ? 6 : N == 32 ? 5 : 4) : N == 16 ? 3 : 2;
    static constexpr int at_q = 2 * ring * tile, at_p = at_q + units * q;
    static constexpr int bytes = at_p + (2 + rests) * p + 1024;
    // From at_p on, of round j: its weights, its rests.
    static __device__ __forceinline__ int weights(int j) { return (j & 1) * p; }
    static __device__ __forceinline__ int rest(int j) { return (rests == 2 ? 2 + (j & 1) : 2) * p; }
    static_assert(bytes <= 227 * 1024 - 4096, "4 KB are for the static part");
};

// The places' shares: the first `more` of `ctas` CTAs have one more than the others.
struct Shares {
    uint32_t each, more;
    __device__ __forceinline__ Shares(uint32_t total, uint32_t ctas) : each(total / ctas), more(total % ctas) {}
    __device__ __forceinline__ uint32_t begin(uint32_t cta) const { return cta * each + min(cta, more); }
    __device__ __forceinline__ uint32_t owner(uint32_t pos) const
    {
        const uint32_t longer = more * (each + 1);
        return pos < longer ? pos / (each + 1) : more + (pos - longer) / each;
    }
};

// Shared-memory descriptor of weights and rests side by side, [key][N columns]: a key's are a line of the 32-, 64- or
// 128-byte swizzle (16-byte piece i of line k is kept at i ^ (k * 2 N / 128 % (N / 8))), 8 lines an atom.  Fields as
// in sw128_desc_mn.
template <int N> __device__ __forceinline__ uint64_t weights_desc(uint32_t saddr)
{
    constexpr uint64_t layout = N == 16 ? 6 : N == 32 ? 4 : 2;
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(8 * 2 * N >> 4) << 32) |
           ((uint64_t)1 << 46) | (layout << 61);
}

template <int DP, int N>
__global__ void __launch_bounds__(kThreads, 1)
paged_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const PagedArgs a)
{
    using S = Smem<DP, N>;
    constexpr int NB = S::ring, QB = S::units, kChunks = N / 16; // stages of keys, of values
    constexpr uint32_t kColumns = N == 16 ? 64 : N == 32 ? 128 : 256;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[2][NB], empty[2][NB], qfull[QB], qempty[QB], sfull[2], pfull[2], pfree[2];
    __shared__ __align__(8) uint64_t ofull, drain;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    __shared__ uint32_t s_sum[kThreads / 32];
    __shared__ Place s_first;
    __shared__ uint32_t s_round[2]; // rounds before this CTA's part, and before its end
    // Of a unit (those of the next ones are made meanwhile): rows' maxima, keys seen, places of the output; keys seen
    // by all rows; which of the keys behind these have values that are no numbers.
    __shared__ __align__(16) float s_m[QB][N];
    __shared__ int s_lim[QB][N];
    __shared__ __nv_bfloat16 *s_out[QB][N];
    __shared__ int s_rows[QB]; // rows that are queries
    __shared__ int s_all[QB];
    __shared__ unsigned long long s_odd[QB];
    __shared__ __align__(16) float s_inv[N], s_scale[N], s_red[4][N];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    asm volatile("griddepcontrol.launch_dependents;");

    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < NB; ++i)
            for (int kv = 0; kv < 2; ++kv) {
                mbar_init(smem_addr(&full[kv][i]), 1);
                mbar_init(smem_addr(&empty[kv][i]), 1);
            }
        for (int i = 0; i < QB; ++i) {
            mbar_init(smem_addr(&qfull[i]), 1);
            mbar_init(smem_addr(&qempty[i]), 5);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sfull[i]), 1);
            mbar_init(smem_addr(&pfull[i]), 4);
            mbar_init(smem_addr(&pfree[i]), 1);
        }
        mbar_init(smem_addr(&ofull), 1);
        mbar_init(smem_addr(&drain), 1);
        abort_s = 0;
        fence_barrier_init();
    }

    // ---- This CTA's part [pos0, pos1) of the sequence; a unit has its rounds' places and kEnd more. ----
    auto block_sum = [&](uint32_t v, uint32_t &before) { // sum over the block; `before`: of the threads before
        uint32_t x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, x, o);
            if (lane >= o)
                x += y;
        }
        if (lane == 31)
            s_sum[warp] = x;
        __syncthreads();
        before = x - v;
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            before += w < warp ? s_sum[w] : 0;
            all += s_sum[w];
        }
        return all;
    };
    uint32_t total = 0, before = 0, mine = 0;
    int rounds = 0, len = 0;
    auto places_of = [&](int b) {
        rounds = b < a.B ? rounds_of(a, b, len) : 0;
        mine = b < a.B ? (uint32_t)((rounds + kEnd) * a.units) : 0;
    };
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        if (b0)
            __syncthreads();
        places_of(b0 + tid);
        total += block_sum(mine, before);
    }
    const uint32_t ctas = min((uint32_t)kCtas, max(1u, total / kMinPlaces)), cta = blockIdx.x;
    if (cta >= ctas)
        return;
    const Shares shares(total, ctas);
    const uint32_t pos0 = shares.begin(cta), pos1 = shares.begin(cta + 1);
    uint32_t run = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        uint32_t all = total;
        if (a.B > kThreads) { // (else the numbers are at hand)
            __syncthreads();
            places_of(b0 + tid);
            all = block_sum(mine, before);
        }
        const uint32_t at = run + before, b = (uint32_t)(b0 + tid);
#pragma unroll
        for (int e = 0; e < 2; ++e) { // this stream has the part's first place; the one behind its last
            const uint32_t pos = e ? pos1 : pos0;
            if (mine > 0 && pos >= at && (pos - at < mine || (e && pos == total && pos - at == mine))) {
                const uint32_t in = pos - at, unit = in / (rounds + kEnd), round = in - unit * (rounds + kEnd);
                s_round[e] = at - kEnd * b * a.units + unit * rounds + min(round, (uint32_t)rounds);
                if (!e)
                    s_first = Place{(int)b, (int)unit, (int)round, rounds, len};
            }
        }
        run += all;
        if (run > pos1)
            break;
    }
    if (warp == 5) {
        tmem_alloc(smem_addr(&tmem_base_s), kColumns);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s, o_col = tmem + 2 * N; // scores: two times N columns
    volatile int *abort = &abort_s;
    Place now = s_first;
    const int count = (int)(s_round[1] - s_round[0]);
    uint32_t unit_pos = pos0 - now.round; // the unit's first place
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
    if (now.round >= now.rounds && count > 0) { // behind a unit's rounds: the next one
        unit_pos += now.rounds + kEnd;
        now.round = now.rounds - 1;
        advance(now);
    }
    auto ends_unit = [&](const Place &p, int j) { return p.round + 1 == p.rounds || j + 1 == count; };

    if (warp == 4 || warp == 7) {
        // ---- Keys (warp 4) and values (warp 7): a box to a lane, its page looked up two rounds ahead, or four rows
        // to a lane, looked up one round ahead.  (Boxes behind the first 32 are looked up as they come: small ones,
        // of pools whose strides have too little in common for the other form.) ----
        constexpr int kSubs = DP / 64;
        const int kv = warp == 7;
        const CUtensorMap *map = kv ? &vmap : &kmap;
        const uint64_t policy = evict_first();
        const int factor = kv ? a.vh : a.kh, boxes = kRound / a.box_rows;
        auto look_up = [&](const Place &p, int box, int &row) { // page and row; a.none (zeros) where there is none
            const int key = p.round * kRound + box * a.box_rows;
            row = 0;
            if (box >= boxes || key >= p.len)
                return a.none;
            const uint32_t page = a.page.div((uint32_t)key);
            row = (int)(key - page * a.page.d);
            return a.table[p.b * a.table_row + page];
        };
        bool ok = true;
        int j = 0;
        auto room = [&]() { // a stage for round j
            if (lane == 0) {
                const int slot = j % NB;
                ok = wait_or_abort(smem_addr(&empty[kv][slot]), ((uint32_t)(j / NB) & 1u) ^ 1u, abort);
                if (ok)
                    mbar_expect_tx(smem_addr(&full[kv][slot]), S::tile);
            }
            ok = __shfl_sync(~0u, ok, 0);
            return ok;
        };
        Place ahead = now; // the round looked up next
        const PagedArgs::Gather &gather = kv ? a.gv : a.gk;
        if (gather.rows) {
            // Lane l has the rows 4 l .. 4 l + 3.
            auto look_up4 = [&](const Place &p, int (&y)[4]) {
                const int head = p.unit / a.tiles * gather.head;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = p.round * kRound + 4 * lane + i;
                    y[i] = 0; // (any row where there is none: it is masked as what lies behind the last token)
                    if (key < p.len) {
                        const uint32_t page = a.page.div((uint32_t)key), e = (uint32_t)a.table[p.b * a.table_row + page];
                        if (e < (uint32_t)a.P)
                            y[i] = (int)e * gather.page + (int)(key - page * a.page.d) * gather.token + head;
                    }
                }
            };
            int y0[4], y1[4];
            look_up4(ahead, y0);
            for (; j < count; ++j) {
                if (j + 1 < count) {
                    advance(ahead);
                    look_up4(ahead, y1);
                }
                if (!room())
                    break;
                const int slot = j % NB;
#pragma unroll
                for (int sub = 0; sub < kSubs; ++sub)
                    tma_gather4_once(base + (kv * NB + slot) * S::tile + sub * S::sub + lane * 512, map, 64 * sub, y0,
                                     smem_addr(&full[kv][slot]), policy);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y0[i] = y1[i];
            }
        } else {
            int page0, row0, page1 = 0, row1 = 0;
            page0 = look_up(ahead, lane, row0);
            if (count > 1) {
                advance(ahead);
                page1 = look_up(ahead, lane, row1);
            }
            for (; j < count; ++j) {
                if (!room())
                    break;
                const int slot = j % NB, head = now.unit / a.tiles * factor;
                const uint32_t bar = smem_addr(&full[kv][slot]), dst = base + (kv * NB + slot) * S::tile;
#pragma unroll 1
                for (int box = lane; box < boxes; box += 32) {
                    if (box >= 32)
                        page0 = look_up(now, box, row0);
                    const int p = (uint32_t)page0 < (uint32_t)a.P ? page0 : a.none;
#pragma unroll
                    for (int sub = 0; sub < kSubs; ++sub)
                        tma_load_4d_once(dst + sub * S::sub + box * a.box_rows * 128, map, 64 * sub, row0, head, p, bar,
                                         policy);
                }
                __syncwarp();
                if (j + 1 < count)
                    advance(now);
                page0 = page1;
                row0 = row1;
                if (j + 2 < count) {
                    advance(ahead);
                    page1 = look_up(ahead, lane, row1);
                }
            }
        }
        if (!ok && lane == 0) // let the copies already issued land before the CTA exits (each wait bounded)
            for (int t = max(0, j - NB); t < j; ++t)
                mbar_wait(smem_addr(&full[kv][t % NB]), (uint32_t)(t / NB) & 1u);
    } else if (warp == 6) {
        // ---- A unit's queries, and what its rows are. ----
        constexpr int kPieces = DP / 8;
        uint32_t u = 0;
        for (int j = 0; j < count; ++u) {
            const int buf = u % QB;
            bool ok = wait_or_abort(smem_addr(&qempty[buf]), ((u / QB) & 1u) ^ 1u, abort);
            ok = __all_sync(~0u, ok);
            if (!ok)
                break;
            const int hk = now.unit / a.tiles, first = (now.unit - hk * a.tiles) * N, rows = a.Nq * a.G;
#pragma unroll 4
            for (int i = lane; i < N * kPieces; i += 32) {
                const int r = i / kPieces, ch = i % kPieces, row = first + r, iq = (int)a.group.div((uint32_t)row);
                const bool have = ch * 8 < a.D && row < rows;
                copy16(base + S::at_q + buf * S::q + (ch >> 3) * (N * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4),
                       have ? a.q.row(now.b, iq, hk * a.G + row - iq * a.G) + ch * 8 : a.q.p, have);
            }
            const int queries = query_count(a, now.b);
#pragma unroll
            for (int r = lane; r < N; r += 32) {
                const int row = first + r, iq = (int)a.group.div((uint32_t)row);
                const bool is = row < rows;
                s_lim[buf][r] = is && iq < queries ? min(max(now.len - queries + iq + 1, 0), now.len) : 0;
                s_out[buf][r] = is ? a.o.row(now.b, iq, hk * a.G + row - iq * a.G) : a.o.p;
            }
            if (lane == 0) {
                // The fewest keys that a row with a token sees; without such rows it is of no account.
                const int iq = (int)a.group.div((uint32_t)first);
                s_all[buf] = iq < queries ? min(max(now.len - queries + iq + 1, 0), now.len) : now.len;
                s_odd[buf] = 0;
                s_rows[buf] = min(N, rows - first);
                if (now.round == 0) {
                    const uint32_t last = unit_pos + now.rounds - 1;
                    a.spans[(int64_t)now.b * a.units + now.unit] =
                        j + now.rounds <= count ? make_int2(-1, -1) : make_int2((int)cta, (int)shares.owner(last));
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&qfull[buf]));
            unit_pos += now.rounds + kEnd;
            j += now.rounds - now.round; // to the next unit
            now.round = now.rounds - 1;
            advance(now);
        }
    } else if (warp == 5) {
        if (lane == 0) {
            const uint32_t idesc_s = idesc_bf16_f32(kRound, N);
            const uint32_t idesc_o = idesc_bf16_f32(DP, S::wide) | kATransposed | kBTransposed;
            const uint64_t kdesc = sw128_desc(base), qdesc = sw128_desc(base + S::at_q);
            const uint64_t vdesc = sw128_desc_mn(base + NB * S::tile, S::sub);
            bool ok = true;
            Place next = now; // of the round whose scores come next
            uint32_t u = 0;
            auto scores = [&](int j) { // s_j = k_j q^T
                const int slot = j % NB;
                ok = wait_or_abort(smem_addr(&qfull[u % QB]), (u / QB) & 1u, abort) &&
                     wait_or_abort(smem_addr(&full[0][slot]), (uint32_t)(j / NB) & 1u, abort);
                if (!ok)
                    return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    umma_bf16(tmem + (j & 1) * N, kdesc + ((slot * S::tile + (k / 4) * S::sub + (k % 4) * 32) >> 4),
                              qdesc + (((u % QB) * S::q + (k / 4) * (N * 128) + (k % 4) * 32) >> 4), idesc_s, k != 0);
                umma_commit(smem_addr(&sfull[j & 1]));
                umma_commit(smem_addr(&empty[0][slot]));
                if (ends_unit(next, j)) {
                    umma_commit(smem_addr(&qempty[u % QB]));
                    ++u;
                }
                if (j + 1 < count)
                    advance(next);
            };
            if (count > 0)
                scores(0);
            bool fresh = true;
            for (int j = 0; j < count && ok; ++j) {
                const Place p = next; // (of round j + 1; where that begins a unit, round j ended one)
                const bool last = j + 1 == count || p.round == 0;
                if (j + 1 < count)
                    scores(j + 1); // (s_(j - 1) has been read: its weights were there)
                const int slot = j % NB;
                ok = ok && wait_or_abort(smem_addr(&full[1][slot]), (uint32_t)(j / NB) & 1u, abort) &&
                     wait_or_abort(smem_addr(&pfull[j & 1]), (uint32_t)(j >> 1) & 1u, abort);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t weights = base + S::at_p + S::weights(j);
                uint64_t pdesc;
                if constexpr (S::split)
                    pdesc = sw128_desc_mn(weights, S::rest(j) - S::weights(j));
                else
                    pdesc = weights_desc<S::wide>(weights);
                // (Leaving out steps of 16 keys behind the last one cost 10% of a long call.)
#pragma unroll
                for (int k = 0; k < kRound / 16; ++k)
                    umma_bf16(o_col, vdesc + ((slot * S::tile + k * 2048) >> 4),
                              pdesc + (k * (16 * S::line) >> 4), idesc_o, !fresh || k > 0);
                umma_commit(smem_addr(&empty[1][slot]));
                umma_commit(smem_addr(&pfree[j & 1]));
                fresh = last;
                if (last)
                    umma_commit(smem_addr(&ofull));
            }
            // Every MMA issued has completed before tensor memory is freed.
            umma_commit(smem_addr(&drain));
            mbar_wait(smem_addr(&drain), 0u);
        }
    } else {
        // ---- Softmax: thread = key. ----
        const uint32_t lanes = (uint32_t)(32 * warp) << 16;
        constexpr bool kHold = N == 16; // a key's scores and what they are relative to stay in registers
        float l[N] = {}, m[kHold ? N : 1];
        const uint32_t pbase = base + S::at_p + tid * S::line;
        const int mix = tid * S::line / 128 % (S::line / 16);
        float *side = a.side + (int64_t)cta * 64 * N;
        bool ok = true, fresh = true, whole = false;
        int all = 0;    // keys that all rows see
        uint32_t u = 0; // units
        int entry = 0;  // of this thread's key, one round ahead; what was where it is none of the stream's
        auto look_up = [&](const Place &p) {
            const int key = p.round * kRound + tid;
            if (key < p.len)
                entry = a.table[p.b * a.table_row + a.page.div((uint32_t)key)];
        };
        look_up(now);
        // No thread leaves before the others know: a wait that has run out shows in the next round's vote.
        for (int j = 0; j < count; ++j) {
            const bool first = fresh;
            const int buf = u % QB;
            auto wait = [&](uint64_t &bar, uint32_t parity) {
                ok = wait_or_abort(smem_addr(&bar), parity & 1u, abort) && ok;
                __syncwarp();
            };
            Place then = now;
            if (fresh) {
                whole = now.round == 0;
                wait(qfull[buf], u / QB);
                all = s_all[buf];
#pragma unroll
                for (int r = 0; r < N; ++r)
                    l[r] = 0.0f;
            }
            const int key = now.round * kRound + tid;
            const bool none = key < now.len && (uint32_t)entry >= (uint32_t)a.P; // a key of no page: its score is no number
            const bool edge = (now.round + 1) * kRound > all; // some row does not see some key
            if (j + 1 < count) {
                advance(then);
                look_up(then);
            }
            wait(sfull[j & 1], (uint32_t)(j >> 1));
            tc_fence_after();
            const uint32_t sc = tmem + (j & 1) * N + lanes;
            float s[16];
            // 16 rows' scores times log2 e less what they are relative to; -inf where the key is not seen.
            auto load = [&](int c, bool absolute) {
                tmem_ld16(sc + 16 * c, s);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const float4 from = absolute ? make_float4(0, 0, 0, 0)
                                        : kHold  ? make_float4(m[kHold ? r : 0], m[kHold ? r + 1 : 0],
                                                               m[kHold ? r + 2 : 0], m[kHold ? r + 3 : 0])
                                                 : *reinterpret_cast<const float4 *>(&s_m[buf][16 * c + r]);
                    s[r] = fmaf(s[r], a.scale2, -from.x);
                    s[r + 1] = fmaf(s[r + 1], a.scale2, -from.y);
                    s[r + 2] = fmaf(s[r + 2], a.scale2, -from.z);
                    s[r + 3] = fmaf(s[r + 3], a.scale2, -from.w);
                }
                if (__builtin_expect(edge || none, 0)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        s[r] = none ? __int_as_float(0x7FC00000) : s[r];
                        s[r] = key < s_lim[buf][16 * c + r] ? s[r] : -INFINITY;
                    }
                }
            };
            auto hold = [&]() {
                if constexpr (kHold) {
#pragma unroll
                    for (int r = 0; r < N; r += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(&s_m[buf][r]);
                        m[r] = x.x;
                        m[r + 1] = x.y;
                        m[r + 2] = x.z;
                        m[r + 3] = x.w;
                    }
                }
            };
            if (first) { // weights are relative to the first key's score, unless another one is far above it
                if (warp == 0) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        load(c, true);
                        if (lane == 0) {
#pragma unroll
                            for (int r = 0; r < 16; ++r)
                                s_m[buf][16 * c + r] = fmaxf(s[r], kLowest);
                        }
                        __syncwarp();
                    }
                }
                softmax_sync();
                hold();
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                load(c, false);
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    top = fmaxf(top, s[r]);
            }
            if (__builtin_expect(softmax_any(top > kGrow || !ok), 0)) {
                if (softmax_any(!ok))
                    break;
                // The rows' maxima over the round's keys and what weights were relative to.
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    load(c, true);
                    const float most = reduce16<true>(s);
                    if (!(lane & 1))
                        s_red[warp][16 * c + (lane >> 1)] = most;
                }
                softmax_sync();
                if (tid < N) {
                    const float most = fmaxf(fmaxf(s_red[0][tid], s_red[1][tid]), fmaxf(s_red[2][tid], s_red[3][tid]));
                    const float from = s_m[buf][tid], to = most > from + kGrow ? most : from;
                    s_m[buf][tid] = to;
                    s_scale[tid] = exp2_fast(from - to); // (of the first round: not used)
                }
                softmax_sync();
                if (!first) { // what is there already is relative to the value before
                    wait(pfree[(j - 1) & 1], (uint32_t)((j - 1) >> 1));
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < S::wide / 16; ++c) {
                        float o[16];
                        tmem_ld16(o_col + lanes + 16 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            o[r] *= s_scale[c % kChunks * 16 + r];
                            if (c < kChunks)
                                l[c % kChunks * 16 + r] *= s_scale[c % kChunks * 16 + r];
                        }
                        tmem_st16(o_col + lanes + 16 * c, o);
                    }
                    tmem_wait_st();
                }
                hold();
                if constexpr (kHold)
                    load(0, false);
            }
            if constexpr (S::rests == 1) { // (the products end in order)
                if (j >= 1)
                    wait(pfree[(j - 1) & 1], (uint32_t)((j - 1) >> 1));
            } else if (j >= 2)
                wait(pfree[j & 1], (uint32_t)((j - 2) >> 1));
            // Values behind the stream's last token are nobody's and meet weights of 0: zeros in their place.  A
            // value that some rows see and others do not also meets such weights: where it is no finite number, its
            // row is taken out, and what it adds to the rows that see it comes at the unit's end.
            bool odd = false;
            if (edge) {
                constexpr int kPieces = DP / 8; // of a row; piece i of row k is kept at i ^ k within its 8
                const int slot = j % NB, begin = now.round * kRound, keys = min(now.len - begin, kRound);
                unsigned char *tile = smem_raw + (base - smem_addr(smem_raw)) + (NB + slot) * S::tile;
                auto piece = [&](int row, int i) {
                    return reinterpret_cast<uint4 *>(tile + (i >> 3) * S::sub + row * 128 + ((i ^ row) & 7) * 16);
                };
                wait(full[1][slot], (uint32_t)(j / NB));
#pragma unroll 4
                for (int i = keys * kPieces + tid; i < kRound * kPieces; i += 128)
                    *piece(i / kPieces, i % kPieces) = make_uint4(0, 0, 0, 0);
                const int some0 = max(all - begin, 0), some = (keys - some0) * kPieces;
                if (some > 0) {
                    bool bad = false;
                    for (int i = tid; i < some; i += 128) {
                        const uint4 x = *piece(some0 + i / kPieces, i % kPieces);
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            bad |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
                    }
                    if (__builtin_expect(softmax_any(bad), 0) && tid >= some0 && tid < keys) {
                        for (int i = 0; i < kPieces; ++i) {
                            const uint4 x = *piece(tid, i);
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                            for (int k = 0; k < 4; ++k)
                                odd |= (w[k] & 0x7F80u) == 0x7F80u || (w[k] & 0x7F800000u) == 0x7F800000u;
                        }
                        if (odd) {
                            for (int i = 0; i < kPieces; ++i)
                                *piece(tid, i) = make_uint4(0, 0, 0, 0);
                            atomicOr(&s_odd[buf], 1ull << (key - all));
                        }
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if constexpr (!kHold)
                    load(c, false);
                if (__builtin_expect(odd, 0)) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        side[(key - all) * N + 16 * c + r] = s[r] + s_m[buf][16 * c + r];
                }
                __syncwarp();
                uint32_t w[16]; // weights, then rests
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    const float e0 = exp2_fast(s[r]), e1 = exp2_fast(s[r + 1]);
                    l[16 * c + r] += e0;
                    l[16 * c + r + 1] += e1;
                    w[r / 2] = pack_bf16x2(e0, e1);
                    w[8 + r / 2] = pack_bf16x2(e0 - bf16_lo(w[r / 2]), e1 - bf16_hi(w[r / 2]));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int piece = (S::split ? 0 : i / 2 * (N / 8)) + 2 * c + i % 2; // of the key's line
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     pbase + (S::split && i >= 2 ? S::rest(j) : S::weights(j)) + ((piece ^ mix) << 4)),
                                 "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                                 : "memory");
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&pfull[j & 1]));
            __syncwarp(); // the arrival goes out before any lane begins to wait
            fresh = ends_unit(now, j);
            if (!fresh) {
                now = then;
                continue;
            }

            // ---- The unit's end, or that of this CTA's part. ----
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                float x[16];
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    x[r] = l[16 * c + r];
                const float sum = reduce16<false>(x);
                if (!(lane & 1))
                    s_red[warp][16 * c + (lane >> 1)] = sum;
            }
            softmax_sync();
            const bool alone = whole && now.round + 1 == now.rounds;
            if (tid < N) {
                // (a row without a token is not masked where all others see the whole round)
                const float sum = s_lim[buf][tid] == 0
                                      ? 0.0f
                                      : (s_red[0][tid] + s_red[1][tid]) + (s_red[2][tid] + s_red[3][tid]);
                s_inv[tid] = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum); // (a sum of NaN gives NaN, no key 0)
                if (!alone)
                    a.stats[(cta * 2 + whole) * N + tid] = make_float2(sum == 0.0f ? -INFINITY : s_m[buf][tid], sum);
                else if (a.lse && tid < s_rows[buf]) {
                    const int hk = now.unit / a.tiles, row = (now.unit - hk * a.tiles) * N + tid;
                    const int iq = (int)a.group.div((uint32_t)row);
                    a.lse[((int64_t)now.b * a.Hq + hk * a.G + row - iq * a.G) * a.Nq + iq] =
                        sum == 0.0f ? -INFINITY : (s_m[buf][tid] + log2f(sum)) * 0.6931471805599453f;
                }
            }
            softmax_sync();
            wait(ofull, u);
            tc_fence_after();
            // (64 channels are 16 lanes of each warp)
            const int d = DP == 128 ? tid : 16 * warp + lane;
            const bool live = d < a.D && (DP == 128 || lane < 16);
            const unsigned long long odds = s_odd[buf];
            const int live_rows = s_rows[buf];
            float *part = a.part + (int64_t)(cta * 2 + whole) * N * a.D + d;
#pragma unroll 1
            for (int c = 0; 16 * c < live_rows; ++c) {
                float o[16];
                float rest[16];
                tmem_ld16(o_col + lanes + 16 * c, o);
                tmem_ld16(o_col + lanes + N + 16 * c, rest);
                tmem_wait_ld();
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    o[r] += fabsf(o[r]) < INFINITY ? rest[r] : 0.0f; // (of an infinite value the rest is no number)
                if (__builtin_expect(odds && live, 0)) {
                    for (unsigned long long left = odds; left; left &= left - 1) {
                        const int at = __ffsll((long long)left) - 1, k = all + at;
                        const uint32_t pg = a.page.div((uint32_t)k);
                        const int e = a.table[now.b * a.table_row + pg];
                        const float v = (uint32_t)e < (uint32_t)a.P
                                            ? __bfloat162float(a.v.row(e, k - pg * a.page.d, now.unit / a.tiles)[d])
                                            : 0.0f;
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (k < s_lim[buf][16 * c + r])
                                o[r] += exp2_fast(side[at * N + 16 * c + r] - s_m[buf][16 * c + r]) * v;
                    }
                }
                if (alone && live) {
#pragma unroll
                    for (int g = 0; g < 16; g += 4) {
                        if (16 * c + g >= live_rows)
                            break;
                        const float4 inv = *reinterpret_cast<const float4 *>(&s_inv[16 * c + g]);
                        const float f[4] = {inv.x, inv.y, inv.z, inv.w};
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (16 * c + g + r < live_rows)
                                s_out[buf][16 * c + g + r][d] = __float2bfloat16_rn(f[r] == 0.0f ? 0.0f : o[g + r] * f[r]);
                        }
                    }
                } else if (live) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        part[(16 * c + r) * a.D] = o[r]; // (of rows that are none, too: nobody reads them)
                }
                __syncwarp();
            }
            tc_fence_before();
            if (lane == 0)
                mbar_arrive(smem_addr(&qempty[buf])); // (this warp is done with the unit's numbers)
            __syncwarp();
            ++u;
            now = then;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, kColumns);
    }
    if (tid == 0 && *abort)
        atomicAdd(&g_paged_timeouts, 1u);
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
    const int2 span = a.spans[(int64_t)b * a.units + hk * a.tiles + row / a.rows];
    if (!span_joins(span.x, span.y, kCtas))
        return;
    const int n = span.y - span.x + 1, r = row % a.rows;
    auto place = [&](int i) { return ((int64_t)(span.x + i) * 2 + (i == 0)) * a.rows + r; }; // (the first begins it)
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
    // Query rows of a unit: 16, 32 or 64.
    int64_t rows() const
    {
        const int64_t r = Nq * (Hq / Hkv);
        return r <= 16 ? 16 : r <= 32 ? 32 : 64;
    }
    int64_t tiles() const { return (Nq * (Hq / Hkv) + rows() - 1) / rows(); }
    int64_t units() const { return Hkv * tiles(); } // of a stream
    int64_t at_stats() const { return (int64_t)kCtas * 2 * rows() * D * 4; }
    int64_t at_side() const { return at_stats() + (int64_t)kCtas * 2 * rows() * 8; }
    int64_t at_spans() const { return at_side() + (int64_t)kCtas * 64 * rows() * 4; }
    int64_t workspace() const { return B == 0 || Nq == 0 ? 0 : at_spans() + B * units() * 8; }
};

template <int DP, int N>
tok_status launch(const CUtensorMap &k, const CUtensorMap &v, const PagedArgs &a, cudaStream_t stream)
{
    const cudaError_t e =
        cudaFuncSetAttribute(paged_kernel<DP, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<DP, N>::bytes);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    paged_kernel<DP, N><<<kCtas, kThreads, Smem<DP, N>::bytes, stream>>>(k, v, a);
    const tok_status st = launch_status();
    return st == TOK_OK ? launch_join(paged_join_kernel, (int64_t)a.B * a.Nq * a.Hq, a, stream) : st;
}

template <int DP>
tok_status launch_rows(const CUtensorMap &k, const CUtensorMap &v, const PagedArgs &a, cudaStream_t stream)
{
    return a.rows == 16   ? launch<DP, 16>(k, v, a, stream)
           : a.rows == 32 ? launch<DP, 32>(k, v, a, stream)
                          : launch<DP, 64>(k, v, a, stream);
}

// Tensor map of a pool with boxes of 64 channels x `rows` tokens; `any`: an address with a row of channels, for a
// pool without pages.
bool pages_map(CUtensorMap *map, const PagesView &x, const void *any, int64_t P, int64_t page_size, int64_t H, int64_t D,
               int rows)
{
    const PoolMap m = pool_map(x, P, page_size, H, D);
    const uint32_t box[4] = {64, (uint32_t)rows, 1, 1};
    return encode_tensor_map_sw128(map, 4, P > 0 ? x.p : any, m.dims, m.strides, box);
}

constexpr int64_t kIntMax = ((int64_t)1 << 31) - 1;

// Tensor map of a pool for copies of four rows: page, token and head as one coordinate, in units of what their
// strides have in common; false (and no rows) where that is less than a row.
bool gather_map(CUtensorMap *map, PagedArgs::Gather *g, const PagesView &x, int64_t P, int64_t page_size, int64_t H, int64_t D)
{
    const int64_t pg = P > 1 ? x.pg : 0, t = page_size > 1 ? x.t : 0, h = H > 1 ? x.h : 0;
    int64_t unit = std::gcd(std::gcd(pg, t), h);
    unit = unit ? unit : (D + 7) / 8 * 8;
    if (unit < D || P < 1 || pg / unit >= kIntMax || t / unit >= kIntMax || h / unit >= kIntMax)
        return false;
    int64_t a, b;
    if (!prod_ok({P - 1, pg / unit}, &a) || !prod_ok({page_size - 1, t / unit}, &b) || a > kIntMax || b > kIntMax)
        return false;
    const int64_t rows = a + b + (H - 1) * (h / unit) + 1;
    if (rows >= kIntMax)
        return false;
    const uint64_t dims[2] = {(uint64_t)D, (uint64_t)rows}, strides[1] = {(uint64_t)unit * 2};
    const uint32_t box[2] = {64, 1};
    *g = {(int)(pg / unit), (int)(t / unit), (int)(h / unit), (int)rows};
    return encode_tensor_map_sw128(map, 2, x.p, dims, strides, box);
}

} // namespace

tok_status read_and_clear_paged_timeouts(cudaStream_t stream, unsigned int *count)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, g_paged_timeouts, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost,
                                              stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && *count)
        e = cudaMemcpyToSymbolAsync(g_paged_timeouts, &zero, sizeof(unsigned int), 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    return TOK_OK;
}

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
    int64_t rounds;
    if (!prod_ok({B, dim.units(), tokens / kRound + 1 + kEnd}, &rounds) || rounds > kIntMax)
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
    a.side = reinterpret_cast<float *>(ws + dim.at_side());
    a.spans = reinterpret_cast<int2 *>(ws + dim.at_spans());
    a.table_row = table_row;
    a.B = (int)B;
    a.Nq = (int)Nq;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.D = (int)D;
    a.rows = (int)dim.rows();
    a.tiles = (int)dim.tiles();
    a.units = (int)dim.units();
    a.P = (int)P;
    a.none = pool_map(a.k, P, page_size, Hkv, D).none; // (the same for both pools)
    a.tokens = (int)tokens;
    a.page = FastDiv((uint32_t)page_size);
    a.group = FastDiv((uint32_t)a.G);
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    a.box_rows = (int)std::min<int64_t>(page_size & -page_size, kRound);
    a.kh = Hkv > 1 && a.k.h == 0 ? 0 : 1;
    a.vh = Hkv > 1 && a.v.h == 0 ? 0 : 1;
    CUtensorMap km, vm;
    // Boxes of 1 or 2 rows are bound by the copies' issue: four rows of any pages to a copy instead (4 streams of
    // 9952 keys, 12 key heads x 96, pages of 1: 258 -> 92 us).  From 4 rows on boxes are no more copies and cost
    // less: 83 us on pages of 4, 56 of 8, 48 of 16.
    if (a.box_rows <= 2) {
        PagedArgs::Gather gk{}, gv{};
        if (gather_map(&km, &gk, a.k, P, page_size, Hkv, D) && gather_map(&vm, &gv, a.v, P, page_size, Hkv, D)) {
            a.gk = gk;
            a.gv = gv;
        }
    }
    if (a.gk.rows == 0 && (!pages_map(&km, a.k, a.q.p, P, page_size, Hkv, D, a.box_rows) ||
        !pages_map(&vm, a.v, a.q.p, P, page_size, Hkv, D, a.box_rows)))
        return TOK_ERR_SHAPE;
    return D <= 64 ? launch_rows<64>(km, vm, a, stream) : launch_rows<128>(km, vm, a, stream);
}
