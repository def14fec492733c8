// What the cross-attention kernels share: the call's tensors, and warp-level matrix
// products on fragments that are loaded straight from global memory.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"
#include "umma.cuh"

namespace tok {

// One [B, N, H, D] tensor: strides in elements, channels dense.
struct HeadsView {
    __nv_bfloat16 *p;
    int64_t b, n, h;
    __device__ __forceinline__ __nv_bfloat16 *row(int64_t ib, int64_t in, int64_t ih) const
    {
        return p + ib * b + in * n + ih * h;
    }
};

struct AttnArgs {
    HeadsView q, k, v, o, go, dq, dk, dv;
    const float *lse_in; // backward
    float *lse;          // [B, Hq, Nq] or null
    float *part;         // split partials
    const int32_t *lens; // [B] or null
    int B, Nq, Nk, Hq, Hkv, G, D;
    int splits;
    float scale, scale2; // scale2 = scale * log2(e)
};

// 2^x, 2 ulp; 0 for -inf.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How many of a grid's equal items run whole: the last, unfull round of the SMs (all of them, where
// there are fewer than SMs) is split into `shares` of an item's `steps` where that is estimated to be
// faster, the shares' partial results being added up by a second kernel.  In us: a step, what
// an item costs around its steps, writing and reading one partial result.
struct Rounds {
    int64_t whole, tail, shares, per; // items whole, items split, shares of each, steps of a share
    Rounds(int64_t items, int64_t steps, int64_t most, double step_us, double item_us, double part_us)
        : whole(items), tail(0), shares(1), per(steps > 0 ? steps : 1)
    {
        constexpr int64_t sms = 148;
        constexpr double join_us = 6; // a second kernel
        const int64_t last = items % sms;
        double best = steps * step_us + item_us;
        for (int64_t s = 2; last > 0 && s <= most && s <= steps; ++s) {
            const int64_t p = (steps + s - 1) / s;
            const double us = (double)((last * s + sms - 1) / sms) * (p * step_us + item_us) + join_us + last * s * part_us;
            if (us < best) {
                best = us;
                whole = items - last;
                tail = last;
                shares = (steps + p - 1) / p; // (none without steps)
                per = p;
            }
        }
    }
};

// The partial results of one query row, `n` of them `stride` rows apart, joined in order by one warp:
// lane s holds the statistics of part s, all lanes 4 channels each.
__device__ __forceinline__ void join_parts(const float *part, const float2 *ml, int64_t stride, int n, int D,
                                           __nv_bfloat16 *o, float *lse)
{
    const int lane = threadIdx.x & 31;
    float ms = -INFINITY, ls = 0.0f;
    if (lane < n) {
        const float2 x = ml[lane * stride];
        ms = x.x;
        ls = x.y;
    }
    float m = ms;
#pragma unroll
    for (int i = 16; i; i >>= 1)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, i));
    const float f = ms == -INFINITY ? ls : exp2_fast(ms - m); // (ls is 0 there, or NaN: no number was the largest)
    float l = f * ls, v[4] = {};
#pragma unroll
    for (int i = 16; i; i >>= 1)
        l += __shfl_xor_sync(~0u, l, i);
    const int d = 4 * lane;
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
        const float fs = __shfl_sync(~0u, f, s);
        if (d < D && fs != 0.0f) { // (a part without keys has written nothing)
            float x[4];
            Row<float, 4, true>::load(part + s * stride * D + d, x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] += fs * x[j];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (d < D) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] *= inv;
        Row<__nv_bfloat16, 4, true>::store(o + d, v);
    }
    if (lane == 0 && lse)
        *lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

constexpr int kMaxSplits = 32; // parts of a query row: a lane of the join each

// A join's CTAs may start while the grid before still runs; they wait for its end (griddepcontrol.wait).
template <class Args> tok_status launch_join(void (*kernel)(Args), int64_t rows, const Args &args, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
    if (e != cudaSuccess) {
        record_cuda_error(e);
        cudaGetLastError();
        return TOK_ERR_CUDA;
    }
    return launch_status();
}

// The forward on the 5th-generation tensor cores (attention_tc.cu): query heads per row tile
// for groups of G, workspace bytes, and the call.  Backward (attention_bwd_tc.cu): likewise.
int attn_tc_group(int G);
int64_t attn_tc_workspace(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D);
tok_status attn_tc_forward(const AttnArgs &a, cudaStream_t stream);
int64_t attn_tc_backward_workspace(int64_t B, int64_t Nq, int64_t Nk, int64_t Hq, int64_t Hkv, int64_t D);
tok_status attn_tc_backward(const AttnArgs &a, float *workspace, cudaStream_t stream);

__device__ __forceinline__ int key_count(const AttnArgs &a, int b)
{
    return a.lens ? min(max(a.lens[b], 0), a.Nk) : a.Nk;
}

// 16 bf16 of a row (8 words), or 8 where only 8 channels are left: whole 32-byte sectors with one store where
// the row is so aligned (`wide`).  A lane stores a row of its own, so a warp's store meets 32 lines
// whatever its width: fewer, wider ones are what counts.
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const uint32_t (&v)[8], int left, bool wide)
{
    if (left <= 0)
        return;
    if (wide && left >= 16) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
        return;
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(v[0], v[1], v[2], v[3]);
    if (left >= 16)
        *reinterpret_cast<uint4 *>(p + 8) = make_uint4(v[4], v[5], v[6], v[7]);
}

// Whether every row of a tensor starts on 32 bytes.
inline bool rows_wide(const HeadsView &v, int64_t B, int64_t N, int64_t H)
{
    return aligned(v.p, 32) && (B <= 1 || v.b % 16 == 0) && (N <= 1 || v.n % 16 == 0) && (H <= 1 || v.h % 16 == 0);
}

// D += A B on one 16 x 8 x 16 tile.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p, bool ok)
{
    return ok ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
}

// Fragments for products over channels (both operands [row][channel]).  The order of a
// contraction is free, so lane c = lane % 4 takes the 16 bytes of channels 32 i + 8 c ..
// + 7 of row lane / 4: its first half is its part of MMA step 2i, the second of 2i + 1.
// chan<NC>: NC = ceil(D / 32) chunks; rows and channels outside are zero.
template <int NC>
__device__ __forceinline__ void load_chan(uint4 (&f)[NC], const __nv_bfloat16 *row, bool ok, int c8, int D)
{
#pragma unroll
    for (int i = 0; i < NC; ++i)
        f[i] = load16(row + 32 * i + c8, ok && 32 * i + c8 < D);
}

// One 16 x 8 tile: rows of lo / hi (lane / 4 and + 8) against the 8 rows of b.
template <int NC>
__device__ __forceinline__ void mma_chan(float (&d)[4], const uint4 (&lo)[NC], const uint4 (&hi)[NC],
                                         const uint4 (&b)[NC])
{
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        mma16816(d, lo[i].x, hi[i].x, lo[i].y, hi[i].y, b[i].x, b[i].y);
        mma16816(d, lo[i].z, hi[i].z, lo[i].w, hi[i].w, b[i].z, b[i].w);
    }
}

// Fragments for products over 16 rows (the B operand is [row][channel], the result's
// columns are channels).  Lane (g = lane / 4, c = lane % 4) takes the 16 bytes of
// channels 64 p + 8 g .. + 7 of rows 2c, 2c + 1, 2c + 8, 2c + 9; column n of tile j is
// channel 64 p + 8 n + j, so a lane's results are the channels 64 p + 16 c + j (and + 8).
struct RowFrag {
    uint4 r[4];
};

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ void mma_rows(float (&acc)[8][4], const uint32_t (&a)[4], const RowFrag &f)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm(word(f.r[0], j / 2), word(f.r[1], j / 2), sel);
        const uint32_t b1 = __byte_perm(word(f.r[2], j / 2), word(f.r[3], j / 2), sel);
        mma16816(acc[j], a[0], a[1], a[2], a[3], b0, b1);
    }
}

__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(~0u, v, 1));
    return fmaxf(v, __shfl_xor_sync(~0u, v, 2));
}
__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor_sync(~0u, v, 1);
    return v + __shfl_xor_sync(~0u, v, 2);
}

// Tensor map of a [B, N, H, D] view with boxes of 64 channels x `heads` x `rows` tokens.
// A dimension of stride 0 becomes one of extent 1 (its coordinate factor is 0).
inline bool heads_map(CUtensorMap *map, const HeadsView &x, int64_t B, int64_t N, int64_t H, int64_t D, int heads, int rows)
{
    auto ext = [](int64_t n, int64_t s) { return (uint64_t)(n > 1 && s == 0 ? 1 : n); };
    auto str = [](int64_t n, int64_t s) { return (uint64_t)(n > 1 && s != 0 ? s * 2 : 16); };
    const uint64_t dims[4] = {(uint64_t)D, ext(H, x.h), ext(N, x.n), ext(B, x.b)};
    const uint64_t strides[3] = {str(H, x.h), str(N, x.n), str(B, x.b)};
    const uint32_t box[4] = {64, (uint32_t)heads, (uint32_t)rows, 1};
    return encode_tensor_map_sw128(map, 4, x.p, dims, strides, box);
}

} // namespace tok
