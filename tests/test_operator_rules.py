"""The token-model operators refuse bad arguments on the host before anything is launched.

No call here reaches a kernel launch: each case fails validation (or is empty) first, so
the tests run on CPU-only machines; the addresses are stand-ins, never dereferenced.
"""
import ctypes

import pytest
import torch

import haar_wavelet_patching_b200 as hwp

F = ctypes.c_void_p
NULL = F(0)
X, Y, TB, POS, BAD = F(0x1000000), F(0x2000000), F(0x3000000), F(0x4000000), F(0x5000000)


@pytest.fixture(scope="module")
def lib():
    from haar_wavelet_patching_b200.build import build
    build()
    return hwp.lib()


def grid(lib, x=X, y=Y, table=TB, dtype=1, B=1, T=2, h=3, w=4, H=2, D=16, xs=(32, 16), ys=(32, 16), o=(0, 0, 0),
         sizes=(2, 3, 4), dims=(4, 4, 8), il=0, f="tok_rope_grid"):
    return getattr(lib, f)(x, y, table, dtype, B, T, h, w, H, D, *xs, *ys, *o, *sizes, *dims, il, NULL)


@pytest.mark.parametrize("f", ["tok_rope_grid", "tok_rope_grid_adjoint"])
def test_rope_grid_rules(lib, f):
    E = hwp
    bad = [dict(dims=(3, 4, 8)), dict(dims=(4, 8, 8)), dict(dims=(-2, 4, 8)), dict(D=15, dims=(4, 4, 6)), dict(B=-1),
           dict(o=(1, 0, 0)), dict(o=(0, -1, 0)), dict(sizes=(2, 3, 3)), dict(ys=(16, 16)), dict(ys=(32, 8)),
           dict(xs=(-32, 16)), dict(B=1 << 30, T=1 << 30), dict(B=1 << 40), dict(w=1 << 62, h=1 << 62)]
    for kw in bad:
        assert grid(lib, f=f, **kw) == E.TOK_ERR_SHAPE, kw
    assert grid(lib, f=f, dtype=2) == E.TOK_ERR_DTYPE
    for kw in (dict(x=NULL), dict(y=NULL), dict(table=NULL)):
        assert grid(lib, f=f, **kw) == E.TOK_ERR_NULL
    assert grid(lib, f=f, x=F(0x1000001)) == E.TOK_ERR_ALIGN
    assert grid(lib, f=f, y=F(0x2000002), dtype=0) == E.TOK_ERR_ALIGN
    assert grid(lib, f=f, table=F(0x3000004)) == E.TOK_ERR_ALIGN
    assert grid(lib, f=f, y=F(0x1000010)) == E.TOK_ERR_ALIAS               # shifted overlap
    assert grid(lib, f=f, y=X, ys=(64, 16)) == E.TOK_ERR_ALIAS             # in place, other strides
    assert grid(lib, f=f, y=F(0x3000000 - 64)) == E.TOK_ERR_ALIAS          # output over the table
    for kw in (dict(B=0), dict(H=0), dict(T=0), dict(D=0, dims=(0, 0, 0))):
        assert grid(lib, f=f, x=NULL, y=NULL, table=NULL, **kw) == E.TOK_OK


def positions(lib, x=X, y=Y, pos=POS, table=TB, bad=BAD, dtype=1, N=5, H=2, D=16, xs=(32, 16), ys=(32, 16),
              sizes=(2, 3, 4), dims=(4, 4, 8), f="tok_rope_positions"):
    return getattr(lib, f)(x, y, pos, table, bad, dtype, N, H, D, *xs, *ys, *sizes, *dims, 0, NULL)


@pytest.mark.parametrize("f", ["tok_rope_positions", "tok_rope_positions_adjoint"])
def test_rope_positions_rules(lib, f):
    assert positions(lib, f=f, N=-1) == hwp.TOK_ERR_SHAPE
    assert positions(lib, f=f, N=1 << 31) == hwp.TOK_ERR_SHAPE
    assert positions(lib, f=f, pos=NULL) == hwp.TOK_ERR_NULL
    assert positions(lib, f=f, pos=F(0x4000002)) == hwp.TOK_ERR_ALIGN
    assert positions(lib, f=f, bad=F(0x5000001)) == hwp.TOK_ERR_ALIGN
    assert positions(lib, f=f, pos=Y) == hwp.TOK_ERR_ALIAS
    assert positions(lib, f=f, bad=Y) == hwp.TOK_ERR_ALIAS
    assert positions(lib, f=f, bad=POS) == hwp.TOK_ERR_ALIAS
    assert positions(lib, f=f, N=0, x=NULL, y=NULL, pos=NULL, table=NULL, bad=NULL) == hwp.TOK_OK


def test_rope_table_rules(lib):
    def table(t=TB, n=(4, 5, 6), d=(4, 2, 2), base=(1e4,) * 3):
        return lib.tok_rope_table(t, *n, *d, *base, 1.0, 1.0, 1.0, NULL)
    for kw in (dict(n=(-1, 5, 6)), dict(d=(3, 2, 2)), dict(base=(1e4, 0.0, 1e4)), dict(base=(float("nan"), 1e4, 1e4)),
               dict(n=(1 << 31, 1, 1)), dict(d=(1 << 17, 2, 2)), dict(n=((1 << 31) - 1, 1, 1), d=(65536, 0, 0))):
        assert table(**kw) == hwp.TOK_ERR_SHAPE, kw
    assert table(t=NULL) == hwp.TOK_ERR_NULL
    assert table(t=F(0x3000004)) == hwp.TOK_ERR_ALIGN
    assert table(t=NULL, n=(0, 0, 0)) == hwp.TOK_OK


def test_rope_binding_refuses():
    x = torch.zeros(1, 2, 3, 4, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.rope_grid(x, torch.zeros(10), (2, 3, 4), (4, 2, 2))
    with pytest.raises(ValueError, match="CUDA"):
        hwp.rope_table((2, 3, 4), (4, 2, 2), device="cpu")
    with pytest.raises(ValueError, match="negative"):
        hwp.rope_table((2, -3, 4), (4, 2, 2))


def sample(lib, x=X, dtype=1, R=4, V=100, stride=100, u=Y, t=NULL, k=NULL, p=NULL, m=NULL, idx=TB, lp=POS):
    return lib.tok_sample_codes(x, dtype, R, V, stride, u, t, 1.0, k, 0, p, 1.0, m, 0.0, idx, lp, NULL)


def test_sample_rules(lib):
    for kw in (dict(R=-1), dict(V=0), dict(V=(1 << 18) + 1), dict(R=(1 << 27) + 1), dict(stride=-1),
               dict(stride=1 << 61)):
        assert sample(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    assert sample(lib, dtype=2) == hwp.TOK_ERR_DTYPE
    for kw in (dict(x=NULL), dict(u=NULL), dict(idx=NULL)):
        assert sample(lib, **kw) == hwp.TOK_ERR_NULL
    for kw in (dict(x=F(0x1000001)), dict(u=F(0x2000002)), dict(t=F(0x5000001)), dict(k=F(0x5000002)),
               dict(p=F(0x5000003)), dict(m=F(0x5000001)), dict(idx=F(0x3000002)), dict(lp=F(0x4000002))):
        assert sample(lib, **kw) == hwp.TOK_ERR_ALIGN
    for kw in (dict(idx=F(0x1000000 + 796)), dict(lp=X), dict(idx=Y), dict(lp=TB), dict(t=TB), dict(k=POS), dict(p=TB),
               dict(m=F(0x3000000 + 12))):
        assert sample(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert sample(lib, R=0, x=NULL, u=NULL, idx=NULL, lp=NULL) == hwp.TOK_OK


def test_sample_binding_refuses():
    with pytest.raises(ValueError, match="CUDA"):
        hwp.sample_codes(torch.zeros(2, 5), torch.zeros(2))


HP = ctypes.POINTER(hwp._Heads)


def heads(addr, strides):
    return ctypes.byref(hwp._Heads(addr, *strides))


Q, K, V, O, LSE, WS = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x60000000
SQ, SK = (4 * 64 * 10, 4 * 64, 64), (2 * 64 * 20, 2 * 64, 64)   # B = 3, Nq = 10, Nk = 20, Hq = 4, Hkv = 2, D = 64


def attend(lib, q=Q, k=K, v=V, o=O, lse=LSE, lens=0, B=3, Nq=10, Nk=20, Hq=4, Hkv=2, D=64, sq=SQ, sk=SK, sv=SK, so=SQ,
           ws=WS, wb=1 << 26):
    return lib.tok_cross_attention(heads(q, sq), heads(k, sk), heads(v, sv), heads(o, so), F(lse), F(lens), B, Nq, Nk, Hq,
                                   Hkv, D, 0.125, F(ws), wb, NULL)


def test_cross_attention_rules(lib):
    for kw in (dict(D=4), dict(D=12), dict(D=136), dict(D=0), dict(Hq=3), dict(Hkv=0), dict(B=-1), dict(Nq=-1), dict(Nk=-1),
               dict(Nq=1 << 30), dict(B=65536), dict(Hq=1 << 17), dict(so=(0, 256, 64)), dict(so=(2560, 256, 32)),
               dict(sk=(2560, -128, 64)), dict(sq=(1 << 40, 256, 64)), dict(B=1, Nq=1, Nk=100000, wb=16), dict(sq=(2560, 0, 64)),
               dict(sq=(2560, 256, 0)), dict(sk=(2560, 0, 64))):
        assert attend(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(B=1, Nq=1, Nk=100000, ws=0)):
        assert attend(lib, **kw) == hwp.TOK_ERR_NULL, kw
    for kw in (dict(q=Q + 8), dict(k=K + 2), dict(o=O + 8), dict(sk=(2560, 132, 64)), dict(lse=LSE + 2), dict(lens=LSE + 1),
               dict(B=1, Nq=1, Nk=100000, ws=WS + 8)):
        assert attend(lib, **kw) == hwp.TOK_ERR_ALIGN, kw
    for kw in (dict(o=Q), dict(o=K), dict(o=Q + 128), dict(o=V - 64), dict(lse=O), dict(lse=Q), dict(lens=LSE),
               dict(B=1, Nq=1, Nk=100000, ws=O), dict(B=1, Nq=1, Nk=100000, ws=K), dict(B=1, Nq=1, Nk=100000, ws=LSE)):
        assert attend(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert attend(lib, B=0, q=0, k=0, v=0, o=0, lse=0) == hwp.TOK_OK
    assert attend(lib, Nq=0, q=0, k=0, v=0, o=0, lse=0) == hwp.TOK_OK
    size = lib.tok_cross_attention_workspace_size
    assert size(1, 1, 8, 3, 2, 64) == -1 and size(1, 1, 8, 2, 2, 65) == -1 and size(0, 1, 8, 2, 2, 64) == 0


def backward(lib, q=Q, k=K, v=V, o=O, lse=LSE, go=0x48000000, lens=0, gq=0x70000000, gk=0x80000000, gv=0x90000000, B=3,
             Nq=10, Nk=20, Hq=4, Hkv=2, D=64, sq=SQ, sgk=SK, sgv=SK, ws=WS, wb=1 << 26):
    return lib.tok_cross_attention_backward(
        heads(q, SQ), heads(k, SK), heads(v, SK), heads(o, SQ), F(lse), heads(go, SQ), F(lens), heads(gq, sq),
        heads(gk, sgk), heads(gv, sgv), B, Nq, Nk, Hq, Hkv, D, 0.125, F(ws), wb, NULL)


def test_cross_attention_backward_rules(lib):
    for kw in (dict(D=20), dict(Hq=5), dict(sgk=(0, 128, 64)), dict(sq=(2560, 200, 64)), dict(wb=64)):
        assert backward(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for kw in (dict(q=0), dict(lse=0), dict(go=0), dict(gq=0), dict(gk=0), dict(gv=0), dict(ws=0)):
        assert backward(lib, **kw) == hwp.TOK_ERR_NULL, kw
    for kw in (dict(gq=0x70000004), dict(ws=WS + 8), dict(lse=LSE + 2)):
        assert backward(lib, **kw) == hwp.TOK_ERR_ALIGN, kw
    fused = (2 * 2560, 256, 64)  # keys' and values' gradients of one [B, Nk, 2, H, D] buffer, overlapping by a head
    for kw in (dict(gq=Q), dict(gk=0x90000000), dict(gv=V), dict(gk=0x70000000), dict(ws=LSE), dict(ws=0x80000000),
               dict(gq=LSE), dict(lens=0x90000000), dict(gk=0x80000000, gv=0x80000000 + 128, sgk=fused, sgv=fused)):
        assert backward(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert backward(lib, B=0, q=0, k=0, v=0, o=0, lse=0, go=0, gq=0, gk=0, gv=0, ws=0) == hwp.TOK_OK


def test_cross_attention_binding_refuses():
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.cross_attention(x, x, x)


def test_cross_attention_spans(lib):
    """Strides that fit each for itself, but whose span over all tokens does not fit into an address."""
    far = dict(B=1, Nq=1, Nk=1 << 29, Hq=1, Hkv=1, wb=1 << 60)
    for s in ((0, 1 << 35, 64), (0, 1 << 37, 64), ((1 << 38) - 8, (1 << 38) - 8, 64)):
        assert attend(lib, sk=s, **far) == hwp.TOK_ERR_SHAPE, s
        assert attend(lib, sv=s, **far) == hwp.TOK_ERR_SHAPE, s
    for s in ((0, 1 << 35, 64), (0, 1 << 37, 64)):
        assert backward(lib, sgk=s, B=1, Nq=1, Nk=1 << 29, Hq=1, Hkv=1, wb=1 << 60) == hwp.TOK_ERR_SHAPE, s
