// Rotary positions of three axes (time, height, width) for the tokens of a latent grid.
//
// Pair i of axis a turns by the angle pos_a * scale_a * base_a^(-2i / d_a):
//   (p, q) -> (p cos - q sin, p sin + q cos),
// the adjoint by the opposite angle.  The R = dt + dh + dw rotated channels of a head are
// the pairs of the three axes in turn, a pair being channels (2i, 2i + 1) (interleaved) or
// (i, i + R / 2); channels past R are copied.
//
// The angles depend on (axis, position, pair) only, so cos and sin come from a table of
// (nt dt + nh dh + nw dw) floats that is made once, in 64 bits (an fp32 angle of position
// 4096 is already 2^-13 off), and stays in L1 / L2: an apply call moves each element once
// in and once out and is bound by HBM.  A thread owns V pairs of one token, reads their
// 2V table values once and turns them in several heads (16-byte loads and stores where
// the layout allows).  Measured: 56,320 tokens x 32 heads (of 48 in a row) x 128, bf16: 146 us,
// 6.3 TB/s; fp32 pairs side by side, 10,395 x 12 x 80: 18 us, 4.4 TB/s (a ramp: 1,625 blocks, less than one round of
// the SMs); 16 tokens: 2 us.
#include <algorithm>
#include <cstdlib>

#include "tma.cuh"
#include "tok_common.cuh"
#include "tok_internal.h"

namespace tok {
namespace {

struct RopeArgs {
    const void *x;
    void *y;
    const float2 *table;
    const int32_t *pos; // [N, 3], or null: the positions are those of the grid
    int32_t *bad_count;
    int64_t xt, xh, yt, yh; // strides in elements: token, head
    int64_t oh, ow;         // float2 offsets of the height and width parts of the table
    FastDiv w, h, t;        // grid extents
    int t0, h0, w0;
    int nt, nh, nw; // table positions
    int pt, ph, P;  // pairs: [0, pt) time, [pt, ph) height, [ph, P) width
    int units, rot_units; // units of V pairs per head: rotated ones, then copied ones (2V channels each)
    FastDiv units_div, groups_div;
    int H, hg; // heads, heads per thread
    uint32_t n0;   // first token of the launch
    uint32_t items; // units * head groups * tokens of the launch
    float sign;
};

// V pairs of one head: registers a[V], b[V].
template <typename T, int V, bool IL> struct Pairs {
    static __device__ __forceinline__ void load(const T *p, int i, int P, float *a, float *b)
    {
        if constexpr (IL) {
            float v[2 * V];
            Row<T, 2 * V, (V > 1)>::load(p + 2 * i, v);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                a[k] = v[2 * k];
                b[k] = v[2 * k + 1];
            }
        } else {
            Row<T, V, (V > 1)>::load(p + i, a);
            Row<T, V, (V > 1)>::load(p + i + P, b);
        }
    }
    static __device__ __forceinline__ void store(T *p, int i, int P, const float *a, const float *b)
    {
        if constexpr (IL) {
            float v[2 * V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                v[2 * k] = a[k];
                v[2 * k + 1] = b[k];
            }
            Row<T, 2 * V, (V > 1)>::store(p + 2 * i, v);
        } else {
            Row<T, V, (V > 1)>::store(p + i, a);
            Row<T, V, (V > 1)>::store(p + i + P, b);
        }
    }
};

constexpr int kThreads = 128; // (256: 153 us instead of 146 on the 16x44x80 grid)

template <typename T, int V, bool IL>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs g)
{
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    if (item >= g.items)
        return;
    // item = (token * groups + group) * units + unit; below 2^31 in a launch.
    const uint32_t tg = g.units_div.div(item);
    const int unit = (int)(item - tg * (uint32_t)g.units);
    const uint32_t ln = g.groups_div.div(tg), n = g.n0 + ln;
    const int h0 = (int)(tg - ln * g.groups_div.d) * g.hg, h1 = h0 + min(g.hg, g.H - h0);
    const T *x = static_cast<const T *>(g.x) + (int64_t)n * g.xt;
    T *y = static_cast<T *>(g.y) + (int64_t)n * g.yt;

    int pt, ph, pw;
    bool ok = true;
    if (g.pos && (unit == 0 || unit < g.rot_units)) { // (unit 0 counts, whether it is rotated or not)
        pt = g.pos[(int64_t)n * 3];
        ph = g.pos[(int64_t)n * 3 + 1];
        pw = g.pos[(int64_t)n * 3 + 2];
        ok = (uint32_t)pt < (uint32_t)g.nt && (uint32_t)ph < (uint32_t)g.nh && (uint32_t)pw < (uint32_t)g.nw;
        if (!ok && unit == 0 && h0 == 0 && g.bad_count)
            atomicAdd(g.bad_count, 1);
    }
    if (unit >= g.rot_units) { // channels that are not rotated
        const int c = 2 * g.P + (unit - g.rot_units) * 2 * V;
        for (int h = h0; h < h1; ++h) {
            float a[V], b[V];
            Row<T, V, (V > 1)>::load(x + h * g.xh + c, a);
            Row<T, V, (V > 1)>::load(x + h * g.xh + c + V, b);
            Row<T, V, (V > 1)>::store(y + h * g.yh + c, a);
            Row<T, V, (V > 1)>::store(y + h * g.yh + c + V, b);
        }
        return;
    }

    if (!g.pos) {
        const uint32_t r = g.w.div(n), q = g.h.div(r), s = g.t.div(q);
        pw = g.w0 + (int)(n - r * g.w.d);
        ph = g.h0 + (int)(r - q * g.h.d);
        pt = g.t0 + (int)(q - s * g.t.d);
    }
    const int i0 = unit * V;
    float c[V], s[V];
    if (ok) {
        const float2 *tt = g.table + (int64_t)pt * g.pt;
        const float2 *th = g.table + g.oh + (int64_t)ph * (g.ph - g.pt) - g.pt;
        const float2 *tw = g.table + g.ow + (int64_t)pw * (g.P - g.ph) - g.ph;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int i = i0 + k;
            const float2 cs = __ldg((i < g.pt ? tt : i < g.ph ? th : tw) + i);
            c[k] = cs.x;
            s[k] = cs.y * g.sign;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            c[k] = s[k] = __int_as_float(0x7FC00000);
    }
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        float a[V], b[V];
        Pairs<T, V, IL>::load(x + h * g.xh, i0, g.P, a, b);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float p = a[k], q = b[k];
            a[k] = fmaf(p, c[k], -(q * s[k]));
            b[k] = fmaf(p, s[k], q * c[k]);
        }
        Pairs<T, V, IL>::store(y + h * g.yh, i0, g.P, a, b);
    }
}

__global__ void rope_table_kernel(float2 *table, int n0, int n1, int n2, int d0, int d1, int d2, double b0, double b1,
                                  double b2, double s0, double s1, double s2, int64_t total)
{
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= total)
        return;
    const int64_t e1 = (int64_t)n0 * (d0 / 2), e2 = e1 + (int64_t)n1 * (d1 / 2);
    const int64_t r = e < e1 ? e : e < e2 ? e - e1 : e - e2;
    const int d = e < e1 ? d0 : e < e2 ? d1 : d2;
    const double base = e < e1 ? b0 : e < e2 ? b1 : b2, scale = e < e1 ? s0 : e < e2 ? s1 : s2;
    const int64_t pos = r / (d / 2);
    const int i = (int)(r - pos * (d / 2));
    double sn, cs;
    sincos((double)pos * scale * pow(base, -2.0 * i / d), &sn, &cs);
    table[e] = make_float2((float)cs, (float)sn);
}

struct RopeCall {
    const void *x;
    void *y;
    const float *table;
    tok_dtype dtype;
    int64_t B, T, h, w; // tokens B * T * h * w (T, h, w: the grid; explicit positions use B = T = h = 1)
    int64_t H, D, xt, xh, yt, yh;
    int64_t t0, h0, w0, nt, nh, nw, dt, dh, dw;
    const int32_t *pos;
    int32_t *bad_count;
    int interleaved;
    bool adjoint;
};

// Bytes from the first to the last element of [n, H, D]; false on overflow or a negative stride.
bool extent(int64_t n, int64_t sn, int64_t H, int64_t sh, int64_t D, int64_t size, int64_t *out)
{
    int64_t a, b, s;
    if (!mul_ok(n - 1, sn, &a) || !mul_ok(H - 1, sh, &b) || __builtin_add_overflow(a, b, &s) ||
        __builtin_add_overflow(s, D, &s))
        return false;
    return mul_ok(s, size, out);
}

template <typename T, int V, bool IL> void launch(const RopeArgs &g, cudaStream_t stream)
{
    rope_kernel<T, V, IL><<<(unsigned)((g.items + kThreads - 1) / kThreads), kThreads, 0, stream>>>(g);
}

template <typename T, bool IL> void launch_v(int v, const RopeArgs &g, cudaStream_t stream)
{
    if (v == 8)
        launch<T, 8, IL>(g, stream);
    else if (v == 4)
        launch<T, 4, IL>(g, stream);
    else if (v == 2)
        launch<T, 2, IL>(g, stream);
    else
        launch<T, 1, IL>(g, stream);
}

tok_status rope_apply(const RopeCall &c, cudaStream_t stream)
{
    constexpr int64_t kMax = (int64_t)1 << 31;
    if (c.dtype != TOK_F32 && c.dtype != TOK_BF16)
        return TOK_ERR_DTYPE;
    const int64_t size = c.dtype == TOK_F32 ? 4 : 2;
    const int64_t R = c.dt + c.dh + c.dw;
    int64_t n, table_floats;
    if (c.dt < 0 || c.dh < 0 || c.dw < 0 || c.dt % 2 || c.dh % 2 || c.dw % 2 || c.D < 0 || c.D % 2 || c.D > 65536 ||
        c.dt > c.D || c.dh > c.D || c.dw > c.D || R > c.D || c.H < 0 || c.H >= kMax || c.nt < 0 || c.nh < 0 ||
        c.nw < 0 || c.nt >= kMax || c.nh >= kMax || c.nw >= kMax || !prod_ok({c.B, c.T, c.h, c.w}, &n) || n >= kMax)
        return TOK_ERR_SHAPE;
    if (!c.pos && (c.t0 < 0 || c.h0 < 0 || c.w0 < 0 || c.t0 > c.nt - c.T || c.h0 > c.nh - c.h || c.w0 > c.nw - c.w))
        return TOK_ERR_SHAPE;
    int64_t ft, fh, fw;
    if (!mul_ok(c.nt, c.dt, &ft) || !mul_ok(c.nh, c.dh, &fh) || !mul_ok(c.nw, c.dw, &fw) ||
        (table_floats = ft + fh + fw) < 0 || table_floats >= kMax * 4)
        return TOK_ERR_SHAPE;
    if (n == 0 || c.H == 0 || c.D == 0)
        return TOK_OK;
    int64_t xb, yb;
    if (c.xt < 0 || c.xh < 0 || c.yt < 0 || c.yh < 0 || !extent(n, c.xt, c.H, c.xh, c.D, size, &xb) ||
        !extent(n, c.yt, c.H, c.yh, c.D, size, &yb) || !nested({{n, c.yt}, {c.H, c.yh}}, c.D))
        return TOK_ERR_SHAPE;
    const bool by_pos = c.pos != nullptr;
    if (!c.x || !c.y || (R > 0 && !c.table))
        return TOK_ERR_NULL;
    if (!aligned(c.x, size) || !aligned(c.y, size) || !aligned(c.table, 8) || !aligned(c.pos, 4) ||
        !aligned(c.bad_count, 4))
        return TOK_ERR_ALIGN;
    // x and y with equal strides are in place, or slices of one buffer whose distance fits into the gaps.
    const bool alike = (n == 1 || c.xt == c.yt) && (c.H == 1 || c.xh == c.yh);
    const int64_t apart = std::abs(((const char *)c.y - (const char *)c.x) / size);
    const bool fits = alike && (apart == 0 || nested({{n, c.yt}, {c.H, c.yh}, {2, apart}}, c.D));
    if ((overlaps(c.x, xb, c.y, yb) && !fits) || overlaps(c.table, table_floats * 4, c.y, yb) ||
        (by_pos && overlaps(c.pos, n * 12, c.y, yb)) ||
        (c.bad_count && (overlaps(c.bad_count, 4, c.y, yb) || overlaps(c.bad_count, 4, c.x, xb) ||
                         overlaps(c.bad_count, 4, c.table, table_floats * 4) ||
                         (by_pos && overlaps(c.bad_count, 4, c.pos, n * 12)))))
        return TOK_ERR_ALIAS;

    // Pairs per thread: the most that the widths, strides and addresses allow as whole
    // vectors of at most 16 bytes (fp32: 4 pairs, bf16: 8).
    const int64_t P = R / 2, rest = c.D - R;
    const bool il = c.interleaved != 0;
    int v = size == 4 ? 4 : 8;
    for (; v > 1; v /= 2) {
        const int64_t vb = std::min<int64_t>(16, (il ? 2 : 1) * v * size), ve = vb / size;
        if (P % v == 0 && rest % (2 * v) == 0 && aligned(c.x, vb) && aligned(c.y, vb) &&
            (n == 1 || (c.xt % ve == 0 && c.yt % ve == 0)) && (c.H == 1 || (c.xh % ve == 0 && c.yh % ve == 0)))
            break;
    }
    RopeArgs g{};
    g.x = c.x;
    g.y = c.y;
    g.table = reinterpret_cast<const float2 *>(c.table);
    g.pos = c.pos;
    g.bad_count = c.bad_count;
    g.xt = c.xt;
    g.xh = c.xh;
    g.yt = c.yt;
    g.yh = c.yh;
    g.oh = c.nt * (c.dt / 2);
    g.ow = g.oh + c.nh * (c.dh / 2);
    g.w = FastDiv((uint32_t)c.w);
    g.h = FastDiv((uint32_t)c.h);
    g.t = FastDiv((uint32_t)c.T);
    g.t0 = (int)c.t0;
    g.h0 = (int)c.h0;
    g.w0 = (int)c.w0;
    g.nt = (int)c.nt;
    g.nh = (int)c.nh;
    g.nw = (int)c.nw;
    g.pt = (int)(c.dt / 2);
    g.ph = (int)((c.dt + c.dh) / 2);
    g.P = (int)P;
    g.rot_units = (int)(P / v);
    g.units = g.rot_units + (int)(rest / (2 * v));
    g.units_div = FastDiv((uint32_t)g.units);
    g.H = (int)c.H;
    // Heads per thread: up to 8 where that still fills the GPU (the table values are read once
    // for all of them; on the 16x44x80 grid with 32 heads 2 cost 5%, 1 costs 27%), fewer for small calls,
    // in equal groups.
    const int64_t threads = n * g.units;
    int64_t hg = std::min<int64_t>(8, c.H);
    while (hg > 1 && threads * ((c.H + hg - 1) / hg) < (int64_t)148 * 1024)
        hg = (hg + 1) / 2;
    hg = (c.H + (c.H + hg - 1) / hg - 1) / ((c.H + hg - 1) / hg);
    int64_t groups = (c.H + hg - 1) / hg;
    while (threads * groups >= kMax && hg < c.H) { // items are 32-bit
        hg = std::min(2 * hg, c.H);
        groups = (c.H + hg - 1) / hg;
    }
    g.hg = (int)hg;
    g.groups_div = FastDiv((uint32_t)groups);
    g.sign = c.adjoint ? -1.0f : 1.0f;
    // (One group where a launch does not hold all tokens; a token has at most 2^15 units then.)
    const int64_t per_token = g.units * groups, most = (kMax - 1) / per_token;
    tok_status st = TOK_OK;
    for (int64_t n0 = 0; n0 < n && st == TOK_OK; n0 += most) {
        g.n0 = (uint32_t)n0;
        g.items = (uint32_t)(std::min(most, n - n0) * per_token);
        if (c.dtype == TOK_F32)
            il ? launch_v<float, true>(v, g, stream) : launch_v<float, false>(v, g, stream);
        else
            il ? launch_v<__nv_bfloat16, true>(v, g, stream) : launch_v<__nv_bfloat16, false>(v, g, stream);
        st = launch_status();
    }
    return st;
}

} // namespace
} // namespace tok

extern "C" tok_status tok_rope_table(float *table, int64_t nt, int64_t nh, int64_t nw, int64_t dt, int64_t dh,
                                     int64_t dw, double base_t, double base_h, double base_w, double scale_t,
                                     double scale_h, double scale_w, cudaStream_t stream)
{
    using namespace tok;
    constexpr int64_t kMax = (int64_t)1 << 31;
    if (nt < 0 || nh < 0 || nw < 0 || nt >= kMax || nh >= kMax || nw >= kMax || dt < 0 || dh < 0 || dw < 0 || dt % 2 ||
        dh % 2 || dw % 2 || dt > 65536 || dh > 65536 || dw > 65536 || !(base_t > 0) || !(base_h > 0) || !(base_w > 0))
        return TOK_ERR_SHAPE;
    const int64_t total = (nt * dt + nh * dh + nw * dw) / 2;
    if (total >= kMax * 2)
        return TOK_ERR_SHAPE;
    if (total == 0)
        return TOK_OK;
    if (!table)
        return TOK_ERR_NULL;
    if (!aligned(table, 8))
        return TOK_ERR_ALIGN;
    rope_table_kernel<<<(unsigned)((total + 127) / 128), 128, 0, stream>>>(
        reinterpret_cast<float2 *>(table), (int)nt, (int)nh, (int)nw, (int)dt, (int)dh, (int)dw, base_t, base_h,
        base_w, scale_t, scale_h, scale_w, total);
    return launch_status();
}

static tok_status rope_grid(bool adjoint, const void *x, void *y, const float *table, tok_dtype dtype, int64_t B,
                            int64_t T, int64_t h, int64_t w, int64_t heads, int64_t D, int64_t x_token,
                            int64_t x_head, int64_t y_token, int64_t y_head, int64_t t0, int64_t h0, int64_t w0,
                            int64_t nt, int64_t nh, int64_t nw, int64_t dt, int64_t dh, int64_t dw, int interleaved,
                            cudaStream_t stream)
{
    const tok::RopeCall c{x,  y,  table, dtype, B,  T,  h,  w,  heads, D,  x_token, x_head,  y_token,     y_head,
                          t0, h0, w0,    nt,    nh, nw, dt, dh, dw,    nullptr, nullptr, interleaved, adjoint};
    return tok::rope_apply(c, stream);
}

static tok_status rope_positions(bool adjoint, const void *x, void *y, const int32_t *pos, const float *table,
                                 int32_t *bad_count, tok_dtype dtype, int64_t N, int64_t heads, int64_t D,
                                 int64_t x_token, int64_t x_head, int64_t y_token, int64_t y_head, int64_t nt,
                                 int64_t nh, int64_t nw, int64_t dt, int64_t dh, int64_t dw, int interleaved,
                                 cudaStream_t stream)
{
    if (!pos && N > 0 && heads > 0 && D > 0)
        return TOK_ERR_NULL;
    static const int32_t none = 0; // an empty call has no positions
    const tok::RopeCall c{x,  y,  table, dtype, 1,  1,  1,  N,  heads, D,  x_token, x_head,  y_token,     y_head,
                          0,  0,  0,     nt,    nh, nw, dt, dh, dw, pos ? pos : &none, bad_count, interleaved, adjoint};
    return tok::rope_apply(c, stream);
}

extern "C" tok_status tok_rope_grid(const void *x, void *y, const float *table, tok_dtype dtype, int64_t B, int64_t T,
                                    int64_t h, int64_t w, int64_t heads, int64_t D, int64_t x_token, int64_t x_head,
                                    int64_t y_token, int64_t y_head, int64_t t0, int64_t h0, int64_t w0, int64_t nt,
                                    int64_t nh, int64_t nw, int64_t dt, int64_t dh, int64_t dw, int interleaved,
                                    cudaStream_t stream)
{
    return rope_grid(false, x, y, table, dtype, B, T, h, w, heads, D, x_token, x_head, y_token, y_head, t0, h0, w0, nt,
                     nh, nw, dt, dh, dw, interleaved, stream);
}

extern "C" tok_status tok_rope_grid_adjoint(const void *gy, void *gx, const float *table, tok_dtype dtype, int64_t B,
                                            int64_t T, int64_t h, int64_t w, int64_t heads, int64_t D,
                                            int64_t gy_token, int64_t gy_head, int64_t gx_token, int64_t gx_head,
                                            int64_t t0, int64_t h0, int64_t w0, int64_t nt, int64_t nh, int64_t nw,
                                            int64_t dt, int64_t dh, int64_t dw, int interleaved, cudaStream_t stream)
{
    return rope_grid(true, gy, gx, table, dtype, B, T, h, w, heads, D, gy_token, gy_head, gx_token, gx_head, t0, h0,
                     w0, nt, nh, nw, dt, dh, dw, interleaved, stream);
}

extern "C" tok_status tok_rope_positions(const void *x, void *y, const int32_t *pos, const float *table,
                                         int32_t *bad_count, tok_dtype dtype, int64_t N, int64_t heads, int64_t D,
                                         int64_t x_token, int64_t x_head, int64_t y_token, int64_t y_head, int64_t nt,
                                         int64_t nh, int64_t nw, int64_t dt, int64_t dh, int64_t dw, int interleaved,
                                         cudaStream_t stream)
{
    return rope_positions(false, x, y, pos, table, bad_count, dtype, N, heads, D, x_token, x_head, y_token, y_head,
                          nt, nh, nw, dt, dh, dw, interleaved, stream);
}

extern "C" tok_status tok_rope_positions_adjoint(const void *gy, void *gx, const int32_t *pos, const float *table,
                                                 int32_t *bad_count, tok_dtype dtype, int64_t N, int64_t heads,
                                                 int64_t D, int64_t gy_token, int64_t gy_head, int64_t gx_token,
                                                 int64_t gx_head, int64_t nt, int64_t nh, int64_t nw, int64_t dt,
                                                 int64_t dh, int64_t dw, int interleaved, cudaStream_t stream)
{
    return rope_positions(true, gy, gx, pos, table, bad_count, dtype, N, heads, D, gy_token, gy_head, gx_token,
                          gx_head, nt, nh, nw, dt, dh, dw, interleaved, stream);
}
