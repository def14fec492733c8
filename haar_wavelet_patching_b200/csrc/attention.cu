// Cross attention to an encoder's states of another length: o = softmax(scale q k^T) v
// over the first len[b] keys of each batch entry, query heads in groups that share a key
// head.  Argument rules, the choice of kernel, and the kernel for few query rows (calls
// with more run on the 5th-generation tensor cores, attention_tc.cu and attention_bwd_tc.cu).
//
// attn_rows_kernel: with few query rows the call is bound by reading the keys and values, so
// it runs on warp-level m16n8k16 tiles.  16 query rows of one key head (queries x the heads of
// its group) per CTA; its 4 warps take 16 keys each in turn with a running maximum and sum of
// their own, joined through shared memory at the end.  Each warp keeps a ring of its own in
// shared memory, all stages but one on their way (cp.async): two CTAs per SM, with 64 KB each in flight
// at 128 channels, cover HBM's latency.  The keys are split over `splits` CTAs; with more than one,
// attn_join_kernel (launched early, it waits for the grid before it) adds up their partial
// results in split order.  Measured: 8 x 1 query, up to 3520 ragged keys, 32 heads on 8, D 128: 20 us,
// of them 5 for the join; its 65 MB take 10 at HBM's rate.
#include <algorithm>

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

// 16 bytes global -> shared, zeros where !ok.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// NP = ceil(D / 64).  Rows of the ring are padded by 16 bytes (value fragments then meet no bank
// conflict, key fragments two-way ones).
template <int NP> struct Ring {
    static constexpr int stages = NP == 2 ? 3 : 4;
    static constexpr int row = NP * 128 + 16, tile = kKeyStep * row; // bytes
    static constexpr int stage = 2 * tile, warp = stages * stage;
    static constexpr int join = kFwdWarps * kRows * NP * 64 * 4; // the warps' results, over the rings
    static constexpr int bytes = kFwdWarps * warp > join ? kFwdWarps * warp : join;
};

__device__ __forceinline__ uint4 shared16(const unsigned char *p) { return *reinterpret_cast<const uint4 *>(p); }

template <int NP>
__global__ void __launch_bounds__(kFwdWarps * 32, 2) attn_rows_kernel(const AttnArgs a)
{
    constexpr int NC = 2 * NP;
    using R = Ring<NP>;
    extern __shared__ __align__(16) unsigned char ring_raw[];
    __shared__ float sm[kFwdWarps][kRows], sl[kFwdWarps][kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int tiles = (a.Nq * a.G + kRows - 1) / kRows;
    const int split = blockIdx.x % a.splits, tile = (int)(blockIdx.x / a.splits) % tiles;
    const int bh = (int)(blockIdx.x / a.splits) / tiles, b = bh / a.Hkv, hk = bh - b * a.Hkv;
    const int rows = a.Nq * a.G, r0 = tile * kRows;
    int k0, k1;
    split_range(key_count(a, b), a.splits, split, k0, k1);
    asm volatile("griddepcontrol.launch_dependents;");

    unsigned char *ring = ring_raw + warp * R::warp;
    const uint32_t ring_s = smem_addr(ring);
    // One step: 16 keys and values, 16 bytes per lane and copy, whole rows together.
    const __nv_bfloat16 *kbase = a.k.row(b, 0, hk), *vbase = a.v.row(b, 0, hk);
    constexpr int kChunks = NP * 8, kCopies = kKeyStep * kChunks / 32; // per tile and lane
    auto fetch = [&](int kk, int stage) {
        const uint32_t dst = ring_s + stage * R::stage;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int e = i * 32 + lane, r = e / kChunks, ch = e % kChunks;
            const bool ok = kk + r < k1 && ch * 8 < a.D;
            const int64_t key = ok ? kk + r : k0;
            const int d = ok ? ch * 8 : 0;
            copy16_async(dst + r * R::row + ch * 16, kbase + key * a.k.n + d, ok);
            copy16_async(dst + R::tile + r * R::row + ch * 16, vbase + key * a.v.n + d, ok);
        }
    };
    constexpr int kRound = kFwdWarps * kKeyStep;
    const int first = k0 + warp * kKeyStep, steps = first < k1 ? (k1 - first + kRound - 1) / kRound : 0;
#pragma unroll
    for (int s = 0; s < R::stages - 1; ++s) {
        if (s < steps)
            fetch(first + s * kRound, s);
        copies_commit();
    }
    uint4 qlo[NC], qhi[NC];
    {
        const int lo = r0 + g, hi = lo + 8;
        load_chan<NC>(qlo, a.q.row(b, lo / a.G, hk * a.G + lo % a.G), lo < rows, 8 * c, a.D);
        load_chan<NC>(qhi, a.q.row(b, hi / a.G, hk * a.G + hi % a.G), hi < rows, 8 * c, a.D);
    }
    float acc[NP][8][4] = {};
    float mlo = -INFINITY, mhi = -INFINITY, llo = 0.0f, lhi = 0.0f;
    for (int step = 0; step < steps; ++step) {
        const int kk = first + step * kRound;
        copies_wait<R::stages - 2>(); // this lane's copies of the step
        __syncwarp();                 // every lane's; and every lane is done with the stage refilled next
        if (step + R::stages - 1 < steps)
            fetch(kk + (R::stages - 1) * kRound, (step + R::stages - 1) % R::stages);
        copies_commit();
        const unsigned char *kt = ring + step % R::stages * R::stage, *vt = kt + R::tile;
        float s[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint4 kf[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i)
                kf[i] = shared16(kt + (8 * t + g) * R::row + 64 * i + 16 * c);
            mma_chan<NC>(s[t], qlo, qhi, kf);
        }
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
        for (int p = 0; p < NP; ++p) {
            RowFrag vf;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                vf.r[i] = shared16(vt + (2 * c + (i & 1) + 8 * (i >> 1)) * R::row + 128 * p + 16 * g);
            mma_rows(acc[p], pa, vf);
        }
    }
    copies_wait<0>();
    __syncthreads(); // every warp is done with its ring: the results go over them
    float(*so)[kRows][NP * 64] = reinterpret_cast<float(*)[kRows][NP * 64]>(ring_raw);
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
    const float inv = l == 0.0f ? 0.0f : 1.0f / l; // (a sum of NaN gives NaN, no key 0)
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
                a.lse[stat] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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
    asm volatile("griddepcontrol.wait;" ::: "memory"); // the grid before has written its parts
    const int64_t nstat = (int64_t)a.B * a.Hq * a.Nq;
    const int64_t stat = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (stat >= nstat)
        return;
    const int iq = (int)(stat % a.Nq), bh = (int)(stat / a.Nq), b = bh / a.Hq, h = bh - b * a.Hq;
    join_parts(a.part + stat * a.D, reinterpret_cast<const float2 *>(a.part + a.splits * nstat * a.D) + stat, nstat,
               a.splits, a.D, a.o.row(b, iq, h), a.lse ? a.lse + stat : nullptr);
}

template <int NP> tok_status launch_rows(const AttnArgs &a, int64_t blocks, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Ring<NP>::bytes);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        return TOK_ERR_CUDA;
    }
    attn_rows_kernel<NP><<<(unsigned)blocks, kFwdWarps * 32, Ring<NP>::bytes, stream>>>(a);
    return launch_status();
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

// Query rows per key head up to which the kernel for few rows takes a call.  Its time grows with every 16 rows, the
// tensor cores' hardly at all (us, few rows / tensor cores, at 48, 64 and 96 rows: 8 x 3520 keys, 32
// heads of 128 on 8: 36 / 38, 45 / 39, 56 / 39; 32 x 300 keys, 16 heads of 64: 22 / 27, 27 / 27, 37 / 27).
constexpr int64_t kTcRows = 48;

bool wants_tc(const Dims &d) { return d.Nq * (d.Hq / d.Hkv) > kTcRows && d.Nk > 0; }

// CTAs that the keys of one 16-row tile are split over.
int64_t rows_splits(const Dims &d)
{
    const int64_t G = d.Hq / d.Hkv;
    // Two CTAs per SM, rounded up to equal splits, each with at least four rounds of its warps (8 x 3520 keys,
    // ragged, 8 key heads: 5 splits, 320 CTAs for the 296 that are resident: 20.0 us; with half as many CTAs 24, twice as many 23; a cluster of 8
    // CTAs that joins through distributed shared memory instead of the workspace: 30).
    const int64_t tiles = (d.Nq * G + kRows - 1) / kRows, units = d.B * d.Hkv * tiles;
    if (units == 0)
        return 1;
    const int64_t want = (148 * 2 + units - 1) / units, most = d.Nk / (4 * kFwdWarps * kKeyStep);
    return std::max<int64_t>(1, std::min(std::min(want, most), (int64_t)kMaxSplits));
}

} // namespace
} // namespace tok

extern "C" int64_t tok_cross_attention_workspace_size(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv,
                                                      int64_t D)
{
    const tok::Dims d{B, Nq, Nk, Hq, Hkv, D};
    if (!d.ok())
        return -1;
    if (tok::wants_tc(d))
        return tok::attn_tc_workspace(B, Nq, Nk, Hq, Hkv, D);
    const int64_t s = tok::rows_splits(d);
    return s > 1 ? s * B * Hq * Nq * (D + 2) * 4 : 0;
}

extern "C" int64_t tok_cross_attention_backward_workspace_size(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq,
                                                               int64_t Hkv, int64_t D)
{
    const tok::Dims d{B, Nq, Nk, Hq, Hkv, D};
    return d.ok() ? tok::attn_tc_backward_workspace(B, Nq, Nk, Hq, Hkv, D) : -1;
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
    const int64_t need = tok_cross_attention_workspace_size(B, Nq, Nk, Hq, Hkv, D);
    const View vq{q, B, Nq, Hq, D, false}, vk{k, B, Nk, Hkv, D, true}, vv{v, B, Nk, Hkv, D, true},
        vo{o, B, Nq, Hq, D, false};
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
    a.scale = scale;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    if (wants_tc(dim))
        return attn_tc_forward(a, stream);
    a.splits = (int)rows_splits(dim);
    const int64_t blocks = B * Hkv * ((Nq * a.G + kRows - 1) / kRows) * a.splits;
    const tok_status st = D <= 64 ? launch_rows<1>(a, blocks, stream) : launch_rows<2>(a, blocks, stream);
    return st == TOK_OK && a.splits > 1 ? launch_join(attn_join_kernel, B * Hq * Nq, a, stream) : st;
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
    const View ins[] = {{q, B, Nq, Hq, D, false}, {o, B, Nq, Hq, D, false}, {grad_o, B, Nq, Hq, D, false},
                        {k, B, Nk, Hkv, D, true}, {v, B, Nk, Hkv, D, true}};
    const View outs[] = {{grad_q, B, Nq, Hq, D, false}, {grad_k, B, Nk, Hkv, D, true}, {grad_v, B, Nk, Hkv, D, true}};
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
    a.lens = k_lens;
    a.B = (int)B;
    a.Nq = (int)Nq;
    a.Nk = (int)Nk;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.D = (int)D;
    a.scale = scale;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    return attn_tc_backward(a, static_cast<float *>(workspace), stream);
}
