// Keys or values in pages: [P, page_size, H, D], strides in elements, channels dense.
#pragma once

#include "attention.cuh"

namespace tok {

struct PagesView {
    __nv_bfloat16 *p;
    int64_t pg, t, h;
    __device__ __forceinline__ __nv_bfloat16 *row(int64_t page, int64_t in, int64_t ih) const
    {
        return p + page * pg + in * t + ih * h;
    }
};

inline PagesView view(const tok_pages *t)
{
    return PagesView{static_cast<__nv_bfloat16 *>(t->ptr), t->page, t->token, t->head};
}

// A pool as the map of the tensor copies has it, innermost first: extents of channels, tokens, heads and pages, byte
// strides of the last three.  Broadcast heads become an extent of 1 (their coordinate factor is 0).  Page `none` lies
// behind the map's last one, so that a copy of it brings zeros and reads nothing.  A pool without pages has no
// element to point at: its map is one row of channels (of the queries), and every copy is one of `none`.
struct PoolMap {
    uint64_t dims[4], strides[3];
    int none;
};

inline PoolMap pool_map(const PagesView &x, int64_t P, int64_t page_size, int64_t H, int64_t D)
{
    if (P <= 0)
        return PoolMap{{(uint64_t)D, 1, 1, 1}, {16, 16, 16}, 1};
    auto str = [](int64_t n, int64_t s) { return (uint64_t)(n > 1 && s != 0 ? s * 2 : 16); };
    return PoolMap{{(uint64_t)D, (uint64_t)page_size, (uint64_t)(x.h == 0 ? 1 : H), (uint64_t)P},
                   {str(page_size, x.t), str(H, x.h), str(P, x.pg)},
                   (int)P};
}

// Whether the CTAs first .. last have written partial results of a unit that are to be joined.  (A CTA that has a
// unit whole leaves a negative number.  Where a wait has run out, units that were not reached have whatever the
// workspace held, which must not be followed: the call has failed, and the join's loads and loops stay within the
// CTAs' places.)
__host__ __device__ constexpr bool span_joins(int first, int last, int ctas)
{
    return first >= 0 && first <= last && last < ctas;
}

// Host: argument rules.
struct PoolView {
    const tok_pages *t;
    int64_t P, N, H, D;
    int64_t span() const
    {
        return (std::max<int64_t>(P, 1) - 1) * t->page + (N - 1) * t->token + (H - 1) * t->head + D;
    }
    bool strides_ok() const
    {
        constexpr int64_t kMax = (int64_t)1 << 38; // elements of one dimension's span: far inside 64 bits as bytes
        for (const Axis &x : {Axis{P, t->page}, Axis{N, t->token}, Axis{H, t->head}})
            if (x.n > 1 && (x.s < 0 || x.s >= kMax / (x.n - 1)))
                return false;
        return (P <= 1 || t->page > 0) && (N <= 1 || t->token > 0);
    }
    bool distinct() const { return nested({{P, t->page}, {N, t->token}, {H, t->head}}, D); }
    bool aligned16() const
    {
        for (const Axis &x : {Axis{P, t->page}, Axis{N, t->token}, Axis{H, t->head}})
            if (x.n > 1 && x.s % 8)
                return false;
        return aligned(t->ptr, 16);
    }
    bool meets(const void *p, int64_t bytes) const { return p && overlaps(t->ptr, span() * 2, p, bytes); }
};

// Whether two pools of the same extents may share an element: their ranges meet, and they are not slices
// that interleave (equal strides, and the distance between them fits into the gaps).
inline bool pools_meet(const PoolView &a, const PoolView &b)
{
    if (!overlaps(a.t->ptr, a.span() * 2, b.t->ptr, b.span() * 2))
        return false;
    if ((a.P > 1 && a.t->page != b.t->page) || (a.N > 1 && a.t->token != b.t->token) ||
        (a.H > 1 && a.t->head != b.t->head))
        return true;
    const int64_t off = ((const char *)b.t->ptr - (const char *)a.t->ptr) / 2;
    return !nested({{a.P, a.t->page}, {a.N, a.t->token}, {a.H, a.t->head}, {2, off < 0 ? -off : off}}, a.D);
}

} // namespace tok
