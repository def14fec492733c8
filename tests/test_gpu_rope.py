"""Rotary positions of three axes against a 64-bit implementation.

Tolerance, from the arithmetic: cos and sin are rounded to fp32 once (2^-24 each), the
product b sin once, the fused multiply-add once, so an fp32 result is within
2^-24 (|a cos| + 2 |b sin| + |y|) <= 4 * 2^-24 (|a| + |b|) of the exact one; a bf16 result
adds half a step, 2^-8 |y| at most (of the rounded value: (1 + 2^-8) covers it).
"""
import numpy as np
import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def angles(pos, dims, base, scale):
    """pos: three float64 tensors [...] -> angles [..., pairs]."""
    out = []
    for a in range(3):
        for i in range(dims[a] // 2):
            out.append(pos[a] * scale[a] * base[a] ** (-2.0 * i / dims[a]))
    return torch.stack(out, -1) if out else pos[0][..., None][..., :0]


def reference(x, pos, dims, interleaved, adjoint=False, base=(1e4,) * 3, scale=(1.0,) * 3):
    """x [..., heads, D] -> exact y and its tolerance, float64."""
    R, D = sum(dims), x.shape[-1]
    th = angles(pos, dims, base, scale)[..., None, :]
    c, s = th.cos(), (-th if adjoint else th).sin()
    f = x.double()
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    ia, ib = ia.to(x.device), ib.to(x.device)
    a, b = f[..., ia], f[..., ib]
    y, tol = f.clone(), torch.zeros_like(f)
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    tol[..., ia] = tol[..., ib] = 4 * U * (a.abs() + b.abs())
    if x.dtype == torch.bfloat16 and R:
        tol[..., ia] += 2.0 ** -8 * (1 + 2.0 ** -8) * y[..., ia].abs()
        tol[..., ib] += 2.0 ** -8 * (1 + 2.0 ** -8) * y[..., ib].abs()
    return y, tol


def grid_positions(T, h, w, origin, device="cuda"):
    return [g.double() for g in torch.meshgrid(*(torch.arange(n, device=device) + o for n, o in zip((T, h, w), origin)),
                                               indexing="ij")]


def check(got, ref, tol, label):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{label}: worst excess {float((err - tol).max()):.3g}"


def randn(*shape, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def test_table_is_exact_to_fp32():
    sizes, dims, base, scale = (5, 9000, 3), (4, 6, 2), (1e4, 500.0, 1e6), (0.5, 1.0, 3.0)
    t = hwp.rope_table(sizes, dims, base, scale).double().cpu()
    at = 0
    for a in range(3):
        n, d = sizes[a], dims[a]
        part = t[at:at + n * d].view(n, d // 2, 2)
        at += n * d
        th = torch.arange(n, dtype=torch.float64)[:, None] * scale[a] * \
            base[a] ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
        # one fp32 rounding (2^-24 of at most 1) and the angle's own 2^-51 of up to 2.7e4
        assert float((part[..., 0] - th.cos()).abs().max()) <= U + 2.0 ** -36
        assert float((part[..., 1] - th.sin()).abs().max()) <= U + 2.0 ** -36


CASES = [  # B, T, h, w, heads, D, dims
    (1, 2, 3, 5, 4, 128, (44, 42, 42)),
    (2, 3, 2, 7, 3, 64, (16, 24, 24)),
    (1, 1, 1, 1, 1, 2, (2, 0, 0)),
    (2, 1, 5, 3, 5, 80, (16, 24, 24)),   # 16 channels copied
    (1, 4, 1, 9, 2, 70, (10, 22, 20)),   # widths that no vector divides
    (1, 2, 2, 2, 3, 6, (0, 2, 0)),
    (1, 2, 2, 2, 3, 8, (0, 0, 0)),       # nothing rotated
    (1, 2, 3, 300, 33, 32, (12, 10, 10)),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_grid(case, interleaved, dtype):
    B, T, h, w, H, D, dims = case
    origin = (2, 0, 1)
    sizes = (T + 2, h, w + 1)
    x = randn(B, T, h, w, H, D, dtype=dtype)
    table = hwp.rope_table(sizes, dims)
    pos = [p.expand(B, T, h, w) for p in grid_positions(T, h, w, origin)]
    for adjoint, f in ((False, hwp.rope_grid), (True, hwp.rope_grid_adjoint)):
        y = f(x, table, sizes, dims, origin=origin, interleaved=interleaved)
        ref, tol = reference(x, pos, dims, interleaved, adjoint)
        check(y, ref, tol, "adjoint" if adjoint else "grid")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,H,D,dims", [(1, 16, 128, (44, 42, 42)), (300, 3, 64, (16, 24, 24)), (77, 1, 10, (4, 2, 2))])
def test_positions(N, H, D, dims, interleaved, dtype):
    sizes = (40, 50, 60)
    x = randn(N, H, D, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.stack([torch.randint(0, n, (N,), generator=g, device="cuda", dtype=torch.int32) for n in sizes], -1)
    table = hwp.rope_table(sizes, dims)
    for adjoint, f in ((False, hwp.rope_positions), (True, hwp.rope_positions_adjoint)):
        y = f(x, pos.contiguous(), table, sizes, dims, interleaved=interleaved)
        ref, tol = reference(x, [pos[:, a].double() for a in range(3)], dims, interleaved, adjoint)
        check(y, ref, tol, "positions")


def test_bad_positions_are_nan_and_counted():
    sizes, dims = (4, 4, 4), (4, 2, 2)
    x = randn(5, 20, 12, dtype=torch.float32)
    pos = torch.tensor([[0, 0, 0], [4, 0, 0], [0, -1, 0], [3, 3, 3], [0, 0, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = hwp.rope_positions(x, pos, hwp.rope_table(sizes, dims), sizes, dims, bad_count=bad)
    assert int(bad) == 3
    nan = y[..., :8].isnan().all(-1).all(-1)
    assert nan.tolist() == [False, True, True, False, True]
    assert torch.equal(y[..., 8:], x[..., 8:]) and not y[[0, 3]].isnan().any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 4])
def test_strides_in_place_and_addresses(interleaved, offset):
    """Slices of a fused projection, odd addresses, in place; nothing beside the slice changes."""
    dims, sizes, H, D = (16, 24, 24), (3, 4, 5), 4, 64
    buf = randn(offset + 60 * (3 * H + 1) * D, dtype=torch.bfloat16)
    rows = buf[offset:].view(1, 3, 4, 5, 3 * H + 1, D)
    x = rows[..., :2 * H, :]
    before = buf.clone()
    table = hwp.rope_table(sizes, dims)
    ref, tol = reference(x, [p[None] for p in grid_positions(3, 4, 5, (0, 0, 0))], dims, interleaved)
    y = hwp.rope_grid(x, table, sizes, dims, interleaved=interleaved)
    assert y.is_contiguous() and torch.equal(buf, before)
    check(y, ref, tol, "strided")
    hwp.tok_rope_grid(x, x, table, sizes, dims, interleaved=interleaved)
    assert torch.equal(x, y)
    rest = before.clone()
    rest[offset:].view_as(rows)[..., :2 * H, :] = y
    assert torch.equal(buf, rest)
    heads_first = torch.empty(1, 2 * H, 3, 4, 5, D, dtype=torch.bfloat16, device="cuda").permute(0, 2, 3, 4, 1, 5)
    rows.copy_(before[offset:].view_as(rows))
    hwp.tok_rope_grid(x, heads_first, table, sizes, dims, interleaved=interleaved)
    assert torch.equal(heads_first, y)


def test_adjoint_is_the_transpose_and_undoes():
    """<rope(x), g> = <x, adjoint(g)>, and the adjoint turns back (rotations are orthogonal)."""
    dims, sizes = (4, 6, 6), (6, 7, 8)
    x, g = randn(2, 6, 7, 8, 3, 20, dtype=torch.float32), randn(2, 6, 7, 8, 3, 20, dtype=torch.float32, seed=2)
    table = hwp.rope_table(sizes, dims)
    y, gx = hwp.rope_grid(x, table, sizes, dims), hwp.rope_grid_adjoint(g, table, sizes, dims)
    lhs, rhs = (y.double() * g.double()).sum(), (x.double() * gx.double()).sum()
    # each element within 4 * 2^-24 (|a| + |b|) of exact: both sums within 8 * 2^-24 sum |x||g| pairwise
    bound = 16 * U * float((x.double().abs().sum() * g.double().abs().max() + g.double().abs().sum() * x.double().abs().max()))
    assert abs(float(lhs - rhs)) <= bound
    back = hwp.rope_grid_adjoint(y, table, sizes, dims)
    a = x.double().abs()
    assert float((back.double() - x.double()).abs().max()) <= 16 * U * float(a.max()) * 2


def test_empty_other_stream_and_graph():
    dims, sizes = (4, 2, 2), (3, 4, 5)
    table = hwp.rope_table(sizes, dims)
    assert hwp.rope_grid(torch.empty(0, 3, 4, 5, 2, 8, device="cuda"), table, sizes, dims).numel() == 0
    assert hwp.rope_positions(torch.empty(0, 2, 8, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                              table, sizes, dims).numel() == 0
    x = randn(1, 3, 4, 5, 2, 8, dtype=torch.float32)
    want = hwp.rope_grid(x, table, sizes, dims)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = hwp.rope_grid(x, table, sizes, dims, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    static, out = x.clone(), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hwp.tok_rope_grid(static, out, table, sizes, dims)
    static.copy_(2 * x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * want)


def test_more_than_2_31_thread_items():
    """A broadcast token turned at every place of a grid of 755 million, three pairs each and no vector that
    divides them (9 GB)."""
    dims, sizes, D = (2, 2, 2), (1024, 1024, 720), 6
    x = randn(1, 1, 1, 1, 1, D, dtype=torch.bfloat16)
    table = hwp.rope_table(sizes, dims)
    y = hwp.rope_grid(x.expand(1, *sizes, 1, D), table, sizes, dims)
    for t in range(0, 1024, 64):
        part = hwp.rope_grid(x.expand(1, 64, *sizes[1:], 1, D), table, sizes, dims, origin=(t, 0, 0))
        assert torch.equal(y[:, t:t + 64], part), t
    tokens = torch.tensor([[0, 0, 0], [970, 1023, 719], [971, 0, 0], [1023, 1023, 719]])
    got = y[0, tokens[:, 0], tokens[:, 1], tokens[:, 2]]
    ref, tol = reference(x[0, 0, 0].expand(4, 1, D), [tokens[:, a].double().cuda() for a in range(3)], dims, False)
    check(got, ref, tol, "far tokens")


@pytest.mark.parametrize("interleaved", [False, True])
def test_into_another_slice_of_the_same_rows(interleaved):
    """Queries of a fused projection turned into its third part: slices of one buffer that share no element."""
    dims, sizes, H, D = (16, 24, 24), (3, 4, 5), 4, 64
    rows = randn(2, 3, 4, 5, 3 * H, D, dtype=torch.bfloat16)
    before = rows.clone()
    x, y = rows[..., :H, :], rows[..., 2 * H:, :]
    table = hwp.rope_table(sizes, dims)
    want = hwp.rope_grid(x.contiguous(), table, sizes, dims, interleaved=interleaved)
    hwp.tok_rope_grid(x, y, table, sizes, dims, interleaved=interleaved)
    assert torch.equal(y, want) and torch.equal(rows[..., : 2 * H, :], before[..., : 2 * H, :])
    rows.copy_(before)  # and the adjoint the other way
    want = hwp.rope_grid_adjoint(y.contiguous(), table, sizes, dims, interleaved=interleaved)
    hwp.tok_rope_grid_adjoint(y, x, table, sizes, dims, interleaved=interleaved)
    assert torch.equal(x, want) and torch.equal(rows[..., H:, :], before[..., H:, :])


def test_bad_positions_are_counted_without_rotated_channels():
    x = randn(4, 3, 8, dtype=torch.float32)
    pos = torch.tensor([[0, 0, 0], [2, 0, 0], [0, -1, 0], [1, 2, 3]], dtype=torch.int32, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = hwp.rope_positions(x, pos, hwp.rope_table((2, 3, 4), (0, 0, 0)), (2, 3, 4), (0, 0, 0), bad_count=bad)
    assert torch.equal(y, x) and int(bad) == 2
