"""Embedding of codes and its gradient against a 64-bit implementation.

Tolerance, from the arithmetic (u = 2^-24; bf16 rounds by at most 2^-8 of the value): y is one fp32 product, u |y|,
and one rounding where it is bf16.  A gradient is a sum of m fp32 terms in some order, at most m u sum|g| off
(first order; the factor 1.01 covers the rest), then one product and one rounding.
"""
import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

U, RB = 2.0 ** -24, 2.0 ** -8 * (1 + 2.0 ** -7)
F32, BF16 = torch.float32, torch.bfloat16


def randn(*shape, dtype=BF16, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def some_codes(N, V, kind, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = (V * torch.rand(N, generator=g, device="cuda", dtype=torch.float64) ** 2).to(torch.int32).clamp_max(V - 1)
    if kind == "hot":
        c = torch.where(torch.rand(N, generator=g, device="cuda") < 0.5, V // 2, c)
    elif kind == "one":
        c = torch.full_like(c, V - 1)
    elif kind == "bad":
        c[::3] = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda").repeat(N)[: len(c[::3])]
    elif kind == "all bad":
        c = torch.full_like(c, -1)
    elif kind == "runs":
        c = (torch.arange(N, device="cuda") // 9).to(torch.int32) % V
    return c.to(torch.int32)


def gradient(g, codes, V, scale, dtype):
    """float64 gradient and its tolerance."""
    codes = codes.flatten().long()
    live = (codes >= 0) & (codes < V)
    rows, codes = g.flatten(0, -2)[live].double(), codes[live]
    z = torch.zeros(V, g.shape[-1], dtype=torch.float64, device="cuda")
    want, mass = z.clone().index_add_(0, codes, rows) * scale, z.index_add_(0, codes, rows.abs()) * abs(scale)
    m = torch.bincount(codes, minlength=V)[:, None]
    tol = 1.01 * U * (m + 2) * mass
    if dtype == BF16:
        tol = tol + RB * (want.abs() + tol)
    return want, tol


def check(got, want, tol, label=""):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{label}: {int((err > tol).sum())} beyond the bound, worst excess {float((err - tol).max()):.3g}"


@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (1, 64000, 2048), (80, 64000, 64), (7, 100, 7), (333, 50, 30), (129, 1000, 4096),
                                   (65, 300, 516), (5000, 64000, 96), (3, 20, 9000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(N, V, D, dtype):
    table, codes = randn(V, D, dtype=dtype), some_codes(N, V, None)
    for scale in (1.0, 0.37):
        want = table.double()[codes.long()] * torch.tensor(scale, dtype=F32).double().item()
        tol = U * want.abs() + (RB * want.abs() if dtype == BF16 else 0)
        check(hwp.embed_codes(codes, table, scale), want, tol)
    assert torch.equal(hwp.embed_codes(codes, table), table[codes.long()])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_forward_rows_and_addresses(dtype, shift):
    """Rows inside larger ones, at every alignment; what lies around them stays."""
    V, D = 40, 24
    big = randn(V, 2 * D + 8, dtype=dtype)
    table = big[:, shift: shift + D]
    codes = some_codes(6, V, None).view(2, 3)
    out = torch.full((2, 3, D + 16), 5.0, dtype=dtype, device="cuda")
    hwp.tok_embed_codes(codes, table, out[..., shift: shift + D])
    assert torch.equal(out[..., shift: shift + D], table[codes.long()])
    assert bool((out[..., :shift] == 5).all()) and bool((out[..., shift + D:] == 5).all())


def test_bad_codes_are_nan_and_counted():
    codes = torch.tensor([3, -1, 10, 0, 2 ** 31 - 1, 9], dtype=torch.int32, device="cuda")
    table, count = randn(10, 2048), torch.zeros(1, dtype=torch.int32, device="cuda")
    y = hwp.embed_codes(codes, table, bad_count=count)
    bad = torch.tensor([1, 2, 4], device="cuda")
    assert count.item() == 3 and bool(y[bad].isnan().all())
    ok = torch.tensor([0, 3, 5], device="cuda")
    assert torch.equal(y[ok], table[codes[ok].long()])


CASES = [(0, 10, 8), (1, 1, 1), (1, 64000, 64), (33, 7, 24), (1000, 1, 129), (5000, 64000, 256), (4097, 300, 2048),
         (20000, 5000, 64), (2048, 1023, 33), (3000, 1024, 40), (3000, 1025, 4096), (70000, 262144, 8)]


@pytest.mark.parametrize("N,V,D", CASES)
@pytest.mark.parametrize("kind", [None, "hot", "one", "bad", "all bad", "runs"])
def test_gradient(N, V, D, kind):
    codes, g = some_codes(N, V, kind), randn(N, D, seed=2)
    want, tol = gradient(g, codes, V, 1.0, BF16)
    got = hwp.embed_codes_backward(g, codes, V)
    check(got, want, tol)
    assert torch.equal(got, hwp.embed_codes_backward(g, codes, V))


@pytest.mark.parametrize("gt,tt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("D", [8, 12, 10, 9, 1004, 3000])
@pytest.mark.parametrize("kind", ["hot", "bad"])
def test_gradient_types_widths_and_scale(gt, tt, D, kind):
    N, V = 3001, 777
    codes, g = some_codes(N, V, kind), randn(N, D, dtype=gt, seed=3)
    want, tol = gradient(g, codes, V, -2.5, tt)
    check(hwp.embed_codes_backward(g, codes, V, scale=-2.5, dtype=tt), want, tol)


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_gradient_rows_workspace_and_surroundings(shift):
    N, V, D = 500, 60, 24
    codes = some_codes(N, V, "hot")
    big = randn(N, 3 * D, seed=4)
    g = big[:, shift: shift + D]
    out = torch.full((V, D + 16), 5.0, dtype=F32, device="cuda")
    need = hwp.embed_codes_backward_workspace_size(N, V, D)
    buf = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    hwp.tok_embed_codes_backward(g, codes, out[:, shift: shift + D], workspace=buf[256: 256 + need])
    want, tol = gradient(g, codes, V, 1.0, F32)
    check(out[:, shift: shift + D], want, tol)
    assert bool((out[:, :shift] == 5).all()) and bool((out[:, shift + D:] == 5).all())
    assert bool((buf[:256] == 77).all()) and bool((buf[256 + need:] == 77).all())
    with pytest.raises(hwp.TokError) as e:
        hwp.tok_embed_codes_backward(g, codes, out[:, :D], workspace=buf[256: 256 + need - 16])
    assert e.value.status == hwp.TOK_ERR_SHAPE


def test_gradient_against_differences():
    """d/dt of sum(w y(table + t dir)) is linear in the table: the difference of two forwards is exact but for roundings."""
    N, V, D = 300, 40, 32
    codes, table, w, d = some_codes(N, V, "hot"), randn(V, D, dtype=F32), randn(N, D, dtype=F32, seed=2), randn(V, D, dtype=F32, seed=3)
    g = hwp.embed_codes_backward(w, codes, V, scale=1.5)
    y1, y0 = hwp.embed_codes(codes, table + d, scale=1.5), hwp.embed_codes(codes, table - d, scale=1.5)
    diff = (w.double() * (y1.double() - y0.double()) / 2).sum()
    slope = (g.double() * d.double()).sum()
    mass = (w.double().abs() * (y1.double().abs() + y0.double().abs())).sum() + (g.double().abs() * d.double().abs()).sum() * N
    assert abs(float(diff - slope)) <= 4 * U * float(mass)


def test_infinities_stay_in_their_rows():
    codes, g = some_codes(200, 30, "hot"), randn(200, 64, dtype=F32)
    g[5], g[9, 3] = float("nan"), float("inf")
    got = hwp.embed_codes_backward(g, codes, 30)
    rows = torch.tensor(sorted({int(codes[5]), int(codes[9])}), device="cuda")
    assert bool(got[int(codes[5])].isnan().all()) and not bool(got[int(codes[9]), 3].isfinite())
    clean = [v for v in range(30) if v not in rows.tolist()]
    assert bool(got[clean].isfinite().all())


def test_streams_graphs_and_empty_calls():
    N, V, D = 4000, 500, 256
    codes, g, table = some_codes(N, V, "hot"), randn(N, D), randn(V, D)
    y, grad = hwp.embed_codes(codes, table), hwp.embed_codes_backward(g, codes, V)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            got.append((hwp.embed_codes(codes, table, stream=s), hwp.embed_codes_backward(g, codes, V, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, y) and torch.equal(b, grad) for a, b in got)
    static = torch.zeros_like(codes)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            y2, grad2 = hwp.embed_codes(static, table), hwp.embed_codes_backward(g, static, V)
        static.copy_(codes)
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(grad2, grad)
    assert hwp.embed_codes(codes[:0], table).shape == (0, D)
    assert bool((hwp.embed_codes_backward(g[:0], codes[:0], V) == 0).all())
    del graph


def test_a_whole_clip():
    """56,320 tokens x 2048 channels: the training step's size, and a table of which most rows stay zero."""
    N, V, D = 56320, 64000, 2048
    codes, g = some_codes(N, V, "hot"), randn(N, D)
    got = hwp.embed_codes_backward(g, codes, V)
    for c0 in range(0, D, 512):
        want, tol = gradient(g[:, c0: c0 + 512], codes, V, 1.0, BF16)
        check(got[:, c0: c0 + 512], want, tol)
