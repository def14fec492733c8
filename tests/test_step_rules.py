"""The operators of a token-by-token step refuse bad arguments on the host before anything is launched.

No call here reaches a kernel launch: each case fails validation (or is empty) first, so
the tests run on CPU-only machines; the addresses are stand-ins, never dereferenced.
"""
import ctypes

import pytest
import torch

import haar_wavelet_patching_b200 as hwp

F = ctypes.c_void_p
NULL = F(0)


def at(n):
    return F(n * 0x10000000)


@pytest.fixture(scope="module")
def lib():
    from haar_wavelet_patching_b200.build import build
    build()
    return hwp.lib()


def embed(lib, codes=at(1), table=at(2), y=at(3), bad=NULL, dtype=1, N=5, V=100, D=64, tr=64, yr=64):
    return lib.tok_embed_codes(codes, table, y, bad, dtype, N, V, D, tr, yr, 1.0, NULL)


def test_embed_rules(lib):
    for kw in (dict(N=-1), dict(N=1 << 30), dict(V=0), dict(V=(1 << 18) + 1), dict(D=0), dict(D=65537), dict(tr=63),
               dict(yr=63), dict(yr=-64), dict(tr=1 << 38), dict(yr=1 << 37)):
        assert embed(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    assert embed(lib, dtype=2) == hwp.TOK_ERR_DTYPE
    for kw in (dict(codes=NULL), dict(table=NULL), dict(y=NULL)):
        assert embed(lib, **kw) == hwp.TOK_ERR_NULL
    for kw in (dict(codes=F(0x10000002)), dict(table=F(0x20000001)), dict(y=F(0x30000002), dtype=0), dict(bad=F(0x50000002))):
        assert embed(lib, **kw) == hwp.TOK_ERR_ALIGN
    for kw in (dict(y=at(2)), dict(y=at(1)), dict(y=F(0x20000000 + 100 * 128 - 2)), dict(bad=at(3)), dict(bad=at(2)),
               dict(bad=at(1))):
        assert embed(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert embed(lib, N=0, codes=NULL, table=NULL, y=NULL) == hwp.TOK_OK


def embed_backward(lib, codes=at(1), g=at(2), t=at(3), gd=1, td=1, N=5, V=100, D=64, gr=64, tr=64, ws=at(4), wb=1 << 27):
    return lib.tok_embed_codes_backward(codes, g, t, gd, td, N, V, D, gr, tr, 1.0, ws, wb, NULL)


def test_embed_backward_rules(lib):
    size = lib.tok_embed_codes_backward_workspace_size
    for kw in (dict(N=-1), dict(N=1 << 30), dict(V=0), dict(V=(1 << 18) + 1), dict(D=0), dict(gr=63), dict(tr=60),
               dict(wb=size(5, 100, 64) - 1)):
        assert embed_backward(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for kw in (dict(gd=2), dict(td=-1)):
        assert embed_backward(lib, **kw) == hwp.TOK_ERR_DTYPE
    for kw in (dict(codes=NULL), dict(g=NULL), dict(t=NULL), dict(ws=NULL)):
        assert embed_backward(lib, **kw) == hwp.TOK_ERR_NULL
    for kw in (dict(codes=F(0x10000002)), dict(g=F(0x20000001)), dict(t=F(0x30000002), td=0), dict(ws=F(0x40000008))):
        assert embed_backward(lib, **kw) == hwp.TOK_ERR_ALIGN
    for kw in (dict(t=at(2)), dict(t=at(1)), dict(t=at(4)), dict(ws=at(2)), dict(ws=at(1))):
        assert embed_backward(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert size(-1, 5, 5) == -1 and size(5, 0, 5) == -1 and size(5, 5, 0) == -1 and size(0, 1, 1) > 0
    for n, v, d in ((0, 1, 1), (1, 64000, 2048), (56320, 64000, 2048), (1 << 29, 1 << 18, 65536)):
        assert size(n, v, d) >= 16 * n


def tables(lib, lens=at(1), fresh=NULL, held=at(2), free=at(3), pages=at(4), table=at(5), slots=at(6), held_out=at(2),
           free_out=at(3), bad=NULL, B=4, N=3, M=7, F_=20, page=16, row=7):
    return lib.tok_page_tables(lens, fresh, held, free, pages, table, slots, held_out, free_out, bad, B, N, M, F_, page,
                               row, NULL)


def test_page_tables_rules(lib):
    for kw in (dict(B=-1), dict(B=65536), dict(N=-1), dict(M=-1), dict(F_=-1), dict(page=0), dict(page=1 << 31), dict(row=6),
               dict(M=1 << 28, row=1 << 28), dict(B=60000, N=1 << 16), dict(F_=1 << 31), dict(row=1 << 37)):
        assert tables(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for name in ("lens", "held", "free", "pages", "table", "slots", "held_out", "free_out"):
        assert tables(lib, **{name: NULL}) == hwp.TOK_ERR_NULL, name
    for i, name in enumerate(("lens", "fresh", "held", "free", "pages", "table", "slots", "held_out", "free_out", "bad")):
        assert tables(lib, **{name: F((i + 9) * 0x10000000 + 2)}) == hwp.TOK_ERR_ALIGN, name
    for kw in (dict(slots=at(5)), dict(slots=at(1)), dict(table=at(4)), dict(held_out=at(1)), dict(held_out=F(0x20000004)),
               dict(free_out=at(2)), dict(bad=at(3)), dict(bad=at(6)), dict(fresh=at(6)), dict(held_out=at(3))):
        assert tables(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert tables(lib, B=0, lens=NULL, held=NULL, free=NULL) == hwp.TOK_OK


def release(lib, lens=at(1), held=at(2), free=at(3), pages=at(4), table=at(5), held_out=at(2), free_out=at(3), bad=NULL,
            B=4, M=7, F_=20, page=16, row=7):
    return lib.tok_page_release(lens, held, free, pages, table, held_out, free_out, bad, B, M, F_, page, row, NULL)


def test_page_release_rules(lib):
    for kw in (dict(B=-1), dict(B=65536), dict(M=-1), dict(F_=-1), dict(page=0), dict(row=6), dict(M=1 << 28, row=1 << 28)):
        assert release(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for name in ("lens", "held", "free", "pages", "table", "held_out", "free_out"):
        assert release(lib, **{name: NULL}) == hwp.TOK_ERR_NULL, name
        assert release(lib, **{name: F(0x90000002)}) == hwp.TOK_ERR_ALIGN, name
    for kw in (dict(pages=at(5)), dict(table=at(1)), dict(held_out=at(1)), dict(free_out=at(4)), dict(bad=at(5))):
        assert release(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert release(lib, B=0, lens=NULL, held=NULL, free=NULL) == hwp.TOK_OK


def heads(addr, strides):
    return ctypes.byref(hwp._Heads(addr, *strides))


def pool(addr, strides):
    return ctypes.byref(hwp._Pages(addr, *strides))


K, V, SL, KP, VP = (n * 0x10000000 for n in range(1, 6))
SK, SP = (3 * 128, 128, 64), (16 * 128, 128, 64)     # B = 4, N = 3, H = 2, D = 64, pages of 16


def write(lib, k=K, v=V, sk=SK, sv=SK, slots=SL, kp=KP, vp=VP, skp=SP, svp=SP, bad=0, B=4, N=3, H=2, D=64, P=10, page=16):
    return lib.tok_paged_write(heads(k, sk), heads(v, sv), F(slots), pool(kp, skp), pool(vp, svp), F(bad), B, N, H, D, P,
                               page, NULL)


def test_paged_write_rules(lib):
    for kw in (dict(B=-1), dict(N=-1), dict(H=0), dict(D=4), dict(D=12), dict(D=136), dict(P=-1), dict(page=0),
               dict(P=1 << 28), dict(B=65536), dict(B=60000, N=1 << 16), dict(sk=(-8, 128, 64)), dict(sk=(384, 0, 64)),
               dict(skp=(2048, 128, 32)), dict(skp=(0, 128, 64)), dict(svp=(2048, 64, 64)), dict(svp=(1 << 38, 128, 64))):
        assert write(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for kw in (dict(k=0), dict(v=0), dict(slots=0), dict(kp=0), dict(vp=0)):
        assert write(lib, **kw) == hwp.TOK_ERR_NULL, kw
    for kw in (dict(k=K + 8), dict(sk=(384, 132, 64)), dict(kp=KP + 8), dict(svp=(2052, 128, 64)), dict(slots=SL + 2),
               dict(bad=SL + 0x8000001)):
        assert write(lib, **kw) == hwp.TOK_ERR_ALIGN, kw
    for kw in (dict(kp=K), dict(vp=KP), dict(vp=KP + 128), dict(kp=SL - 16), dict(bad=KP), dict(bad=SL), dict(bad=K)):
        assert write(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert write(lib, B=0, k=0, v=0, slots=0, kp=0, vp=0) == hwp.TOK_OK
    assert write(lib, N=0, k=0, v=0, slots=0, kp=0, vp=0) == hwp.TOK_OK


Q, O, TB, KL, QL, LSE, WS = (n * 0x10000000 for n in range(6, 13))
SQ = (2 * 256, 256, 64)                                # Nq = 2, Hq = 4


def attend(lib, q=Q, kp=KP, vp=VP, table=TB, kl=KL, ql=0, o=O, lse=LSE, sq=SQ, so=SQ, skp=SP, svp=SP, B=4, Nq=2, Hq=4,
           Hkv=2, D=64, P=10, page=16, M=5, row=5, ws=WS, wb=1 << 27):
    return lib.tok_paged_attention(heads(q, sq), pool(kp, skp), pool(vp, svp), F(table), F(kl), F(ql), heads(o, so),
                                   F(lse), B, Nq, Hq, Hkv, D, P, page, M, row, 0.125, F(ws), wb, NULL)


def test_paged_attention_rules(lib):
    size = lib.tok_paged_attention_workspace_size
    for kw in (dict(D=4), dict(D=12), dict(D=136), dict(Hq=3), dict(Hkv=0), dict(B=-1), dict(Nq=-1), dict(Nq=65),
               dict(B=65536), dict(Hq=1 << 17), dict(P=-1), dict(M=-1), dict(page=0), dict(P=1 << 28), dict(M=1 << 28, row=1 << 28),
               dict(row=4), dict(so=(0, 256, 64)), dict(so=(512, 256, 32)), dict(sq=(512, 0, 64)), dict(skp=(-16, 128, 64)),
               dict(svp=(1 << 38, 128, 64)), dict(wb=size(4, 2, 4, 2, 64) - 1)):
        assert attend(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    for kw in (dict(q=0), dict(kp=0), dict(vp=0), dict(table=0), dict(kl=0), dict(o=0), dict(ws=0)):
        assert attend(lib, **kw) == hwp.TOK_ERR_NULL, kw
    for kw in (dict(q=Q + 8), dict(o=O + 2), dict(kp=KP + 8), dict(svp=(2052, 128, 64)), dict(table=TB + 2), dict(kl=KL + 1),
               dict(ql=QL + 2), dict(lse=LSE + 2), dict(ws=WS + 8)):
        assert attend(lib, **kw) == hwp.TOK_ERR_ALIGN, kw
    for kw in (dict(o=Q), dict(o=KP), dict(o=VP + 128), dict(o=TB), dict(o=KL), dict(ql=O), dict(lse=Q), dict(lse=O),
               dict(lse=KP), dict(lse=TB), dict(ws=Q), dict(ws=O), dict(ws=VP), dict(ws=TB), dict(ws=KL), dict(ws=LSE)):
        assert attend(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert attend(lib, B=0, q=0, kp=0, vp=0, table=0, kl=0, o=0, lse=0, ws=0, wb=0) == hwp.TOK_OK
    assert attend(lib, Nq=0, q=0, kp=0, vp=0, table=0, kl=0, o=0, lse=0, ws=0, wb=0) == hwp.TOK_OK
    assert size(1, 1, 3, 2, 64) == -1 and size(1, 65, 2, 2, 64) == -1 and size(0, 1, 2, 2, 64) == 0 and size(3, 0, 2, 2, 64) == 0


def verify(lib, x=at(1), d=at(2), dtype=1, codes=at(3), u=at(4), n=NULL, t=NULL, out=at(5), acc=at(6), B=4, K=3, V=100,
           lb=400, lr=100, db=300, dr=100, ws=at(7), wb=1 << 27):
    return lib.tok_verify_codes(x, d, dtype, codes, u, n, t, 1.0, out, acc, B, K, V, lb, lr, db, dr, ws, wb, NULL)


def test_verify_rules(lib):
    for kw in (dict(B=-1), dict(B=(1 << 20) + 1), dict(K=-1), dict(K=64), dict(V=0), dict(V=(1 << 18) + 1), dict(lb=-1),
               dict(lr=-1), dict(db=1 << 40), dict(dr=-100), dict(wb=lib.tok_verify_codes_workspace_size(4, 3, 100) - 1)):
        assert verify(lib, **kw) == hwp.TOK_ERR_SHAPE, kw
    assert verify(lib, dtype=2) == hwp.TOK_ERR_DTYPE
    for kw in (dict(x=NULL), dict(codes=NULL), dict(u=NULL), dict(out=NULL), dict(acc=NULL), dict(ws=NULL)):
        assert verify(lib, **kw) == hwp.TOK_ERR_NULL
    for i, name in enumerate(("x", "d", "codes", "u", "n", "t", "out", "acc", "ws")):
        assert verify(lib, **{name: F((i + 9) * 0x10000000 + 1)}) == hwp.TOK_ERR_ALIGN, name
    for kw in (dict(out=at(1)), dict(out=at(2)), dict(out=at(3)), dict(acc=at(4)), dict(acc=at(5)), dict(n=at(6)),
               dict(t=at(5)), dict(ws=at(1)), dict(ws=at(3)), dict(ws=at(5)), dict(ws=at(6))):
        assert verify(lib, **kw) == hwp.TOK_ERR_ALIAS, kw
    assert verify(lib, B=0, x=NULL, d=NULL, codes=NULL, u=NULL, out=NULL, acc=NULL, ws=NULL, wb=0) == hwp.TOK_OK
    size = lib.tok_verify_codes_workspace_size
    assert size(1, 64, 5) == -1 and size(-1, 1, 5) == -1 and size(1, 1, 0) == -1 and size(0, 3, 5) == 0 and size(2, 3, 5) > 0


def test_bindings_refuse():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.embed_codes(torch.zeros(3, **i32), torch.zeros(5, 8))
    with pytest.raises(ValueError, match="CUDA"):
        hwp.embed_codes_backward(torch.zeros(3, 8), torch.zeros(3, **i32), 5)
    one = torch.zeros(1, **i32)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.page_tables(one, None, 4, one, one, one, torch.zeros(1, 3, **i32), 16)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.page_release(one, one, one, one, torch.zeros(1, 3, **i32), 16)
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.paged_write(x, x, x, x, torch.zeros(1, 2, **i32))
    with pytest.raises(ValueError, match="CUDA"):
        hwp.paged_attention(x, x, x, torch.zeros(1, 3, **i32), one)
    with pytest.raises(ValueError, match="CUDA"):
        hwp.verify_codes(torch.zeros(1, 2, 5), torch.zeros(1, 1, **i32), torch.zeros(1, 2))
