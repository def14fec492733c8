"""Cross attention and its gradients against a 64-bit implementation.

Tolerance, from the arithmetic (u = 2^-24; bf16 rounds by at most 2^-8 of the value):
  scores     products of bf16 are exact in fp32, D of them accumulate, so a score (times
             log2 e) is within S = 2 (D + 4) u max sum|q k| |scale| log2 e of the exact one
             (a factor 2 for the accumulator's internal rounding).
  weights    p = 2^(s - m) / l is within a relative E = 2 S + 2^-21 of the exact one (the
             2-ulp power, the sum and the quotient); with the forward's lse in the place of
             m and l, E + 4 u |lse| log2 e.  As an operand it is rounded once, 2^-8.
  underflow  the power gives 0 for results below 2^-126, so a weight is also off by up to 2^-126
             (TINY); a bf16 operand below 2^-126 rounds by at most 2^-134, which TINY covers too.
  o          sum p |v| (2^-8 + E + 2 Nk u), then one rounding of o.
  delta      rowsum(go o) takes the rounded o: sum |go| tol(o) + 2 D u sum |go o|.
  ds         p |dp - delta| (2^-8 + E) + p (2 D u sum |go v| + tol(delta)).
  dq, dk, dv sums of the above against |k|, |q|, |go|, 2 N u of their magnitude for the
             accumulation over N terms, and one rounding.
"""
import math

import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

U, RB = 2.0 ** -24, 2.0 ** -8 * (1 + 2.0 ** -7)
L2E = 1.4426950408889634
TINY = 2.0 ** -126


def randn(*shape, seed=1, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * spread).to(torch.bfloat16)


def reference(q, k, v, lens, scale, go=None):
    """float64 results and tolerances: {name: (value, tol)}."""
    B, Nq, Hq, D = q.shape
    Nk, Hkv = k.shape[1:3]
    G = Hq // Hkv
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    r = {"o": (z(B, Nq, Hq, D), z(B, Nq, Hq, D)), "lse": (z(B, Hq, Nq), z(B, Hq, Nq))}
    if go is not None:
        r.update(dq=(z(B, Nq, Hq, D), z(B, Nq, Hq, D)), dk=(z(B, Nk, Hkv, D), z(B, Nk, Hkv, D)),
                 dv=(z(B, Nk, Hkv, D), z(B, Nk, Hkv, D)))
    for b in range(B):
        n = Nk if lens is None else max(0, min(Nk, int(lens[b])))
        for h in range(Hq):
            j = h // G
            if n == 0:
                r["lse"][0][b, h] = -math.inf
                continue
            qq, kk, vv = q[b, :, h].double(), k[b, :n, j].double(), v[b, :n, j].double()
            s = scale * qq @ kk.T
            S = 2 * (D + 4) * U * abs(scale) * L2E * (qq.abs() @ kk.abs().T).amax(1, keepdim=True)
            lse = torch.logsumexp(s, 1, keepdim=True)
            p = (s - lse).exp()
            E = 2 * S + 2.0 ** -21
            o = p @ vv
            to = (p @ vv.abs()) * (RB + E + 2 * n * U) + RB * o.abs() + TINY * vv.abs().sum(0)
            r["o"][0][b, :, h], r["o"][1][b, :, h] = o, to
            r["lse"][0][b, h], r["lse"][1][b, h] = lse[:, 0], (E + 4 * U * lse.abs() + 2 * n * U)[:, 0]
            if go is None:
                continue
            E = E + 4 * U * lse.abs() * L2E + 2 * n * U
            gg = go[b, :, h].double()
            dp, delta = gg @ vv.T, (gg * o).sum(1, keepdim=True)
            td = (gg.abs() * to).sum(1, keepdim=True) + 2 * D * U * (gg * o).abs().sum(1, keepdim=True)
            ds = p * (dp - delta)
            tds = ds.abs() * (RB + E) + TINY * (1 + (dp - delta).abs()) + p * (2 * D * U * (gg.abs() @ vv.abs().T) + td)
            r["dq"][0][b, :, h] = scale * ds @ kk
            r["dq"][1][b, :, h] = abs(scale) * (tds + 2 * n * U * ds.abs()) @ kk.abs()
            r["dk"][0][b, :n, j] += scale * ds.T @ qq
            r["dk"][1][b, :n, j] += abs(scale) * (tds + 2 * G * Nq * U * ds.abs()).T @ qq.abs()
            r["dv"][0][b, :n, j] += p.T @ gg
            r["dv"][1][b, :n, j] += (p * (RB + E + 2 * G * Nq * U) + TINY).T @ gg.abs()
    for name in ("dq", "dk", "dv"):
        if name in r:
            r[name] = (r[name][0], r[name][1] + RB * r[name][0].abs())
    return r


def check(got, ref, name):
    want, tol = ref[name]
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), f"{name}: infinities differ"
    err = (got - want).abs()[fine]
    tol = tol[fine]
    assert bool((err <= tol + 1e-37).all()), \
        f"{name}: {int((err > tol).sum())} of {err.numel()} beyond the bound, worst {float((err / (tol + 1e-37)).max()):.3g} times it"


def lens_of(kind, B, Nk):
    if kind is None:
        return None
    return torch.tensor({"ragged": [max(0, Nk - 1 - i * (Nk // 2)) for i in range(B)],
                         "empty": [0 if i % 2 == 0 else Nk for i in range(B)],
                         "wild": [(-5, Nk + 7, 1, Nk // 2)[i % 4] for i in range(B)]}[kind],
                        dtype=torch.int32, device="cuda")


FORWARD = [  # B, Nq, Nk, Hq, Hkv, D, lens
    (1, 1, 1, 1, 1, 8, None), (2, 1, 1, 2, 1, 64, "empty"), (3, 1, 513, 8, 2, 128, "ragged"),
    (2, 1, 5000, 32, 8, 128, None), (1, 1, 40001, 1, 1, 64, None), (4, 3, 700, 6, 2, 80, "wild"),
    (2, 17, 33, 3, 3, 40, "ragged"), (1, 128, 128, 2, 2, 64, None), (1, 129, 127, 2, 1, 128, None),
    (2, 300, 385, 4, 4, 96, "ragged"), (3, 257, 130, 4, 2, 128, "wild"), (1, 1000, 640, 4, 4, 64, None),
    (2, 255, 1, 2, 2, 128, None), (1, 515, 1030, 3, 1, 120, None), (5, 200, 260, 2, 2, 56, "wild"),
    (1, 5, 0, 2, 2, 64, None), (2, 300, 0, 2, 2, 128, None), (4, 400, 257, 8, 2, 72, "empty"),
    (1, 700, 129, 16, 1, 128, None), (2, 128, 256, 2, 2, 128, None), (1, 256, 2048, 2, 2, 128, None),
    # a last round of the SMs that is shared: forward, both backward passes
    (1, 2437, 1500, 16, 16, 128, None), (2, 1300, 900, 16, 4, 64, "ragged"), (3, 700, 2100, 18, 18, 80, "wild"),
]


@pytest.mark.parametrize("case", FORWARD)
def test_forward(case):
    B, Nq, Nk, Hq, Hkv, D, kind = case
    q, k, v = randn(B, Nq, Hq, D), randn(B, Nk, Hkv, D, seed=2), randn(B, Nk, Hkv, D, seed=3)
    lens = lens_of(kind, B, Nk)
    ref = reference(q, k, v, lens, D ** -0.5)
    o, lse = hwp.cross_attention(q, k, v, lens, with_lse=True)
    check(o, ref, "o")
    check(lse, ref, "lse")
    assert torch.equal(hwp.cross_attention(q, k, v, lens), o)
    hwp.tok_check_device()


@pytest.mark.parametrize("case", FORWARD)
def test_backward(case):
    B, Nq, Nk, Hq, Hkv, D, kind = case
    q, k, v = randn(B, Nq, Hq, D), randn(B, Nk, Hkv, D, seed=2), randn(B, Nk, Hkv, D, seed=3)
    go = randn(B, Nq, Hq, D, seed=4)
    lens = lens_of(kind, B, Nk)
    ref = reference(q, k, v, lens, D ** -0.5, go)
    o, lse = hwp.cross_attention(q, k, v, lens, with_lse=True)
    first = hwp.cross_attention_backward(q, k, v, o, lse, go, lens)
    for g, name in zip(first, ("dq", "dk", "dv")):
        check(g, ref, name)
    for a, b in zip(first, hwp.cross_attention_backward(q, k, v, o, lse, go, lens)):
        assert torch.equal(a, b)  # every sum has a fixed order
    hwp.tok_check_device()


@pytest.mark.parametrize("Nq,D", [(1, 128), (300, 64), (300, 128), (40, 80)])
def test_masked_places_hold_anything(Nq, D):
    """NaN and infinities behind the lengths reach neither results nor gradients."""
    B, Nk, H = 3, 300, 2
    q, k, v, go = (randn(B, n, H, D, seed=s) for n, s in ((Nq, 1), (Nk, 2), (Nk, 3), (Nq, 4)))
    lens = torch.tensor([129, 0, 250], dtype=torch.int32, device="cuda")
    ref = reference(q, k, v, lens, D ** -0.5, go)
    for b, n in enumerate(lens.tolist()):
        k[b, n:] = math.nan
        v[b, n:] = math.inf
        v[b, n::2] = math.nan
    o, lse = hwp.cross_attention(q, k, v, lens, with_lse=True)
    check(o, ref, "o")
    check(lse, ref, "lse")
    for g, name in zip(hwp.cross_attention_backward(q, k, v, o, lse, go, lens), ("dq", "dk", "dv")):
        check(g, ref, name)
    assert bool((hwp.cross_attention_backward(q, k, v, o, lse, go, lens)[1][1] == 0).all())


@pytest.mark.parametrize("Nq", [2, 260])
@pytest.mark.parametrize("spread,scale", [(8.0, None), (1.0, 2.0), (1.0, -0.3), (1.0, 0.0), (30.0, 1.0)])
def test_large_scores_and_other_scales(Nq, spread, scale):
    B, Nk, H, D = 1, 400, 2, 64
    q, k, v, go = (randn(B, n, H, D, seed=s, spread=f) for n, s, f in
                   ((Nq, 1, spread), (Nk, 2, spread), (Nk, 3, 1.0), (Nq, 4, 1.0)))
    sc = D ** -0.5 if scale is None else scale
    ref = reference(q, k, v, None, sc, go)
    o, lse = hwp.cross_attention(q, k, v, scale=scale, with_lse=True)
    check(o, ref, "o")
    check(lse, ref, "lse")
    for g, name in zip(hwp.cross_attention_backward(q, k, v, o, lse, go, scale=scale), ("dq", "dk", "dv")):
        check(g, ref, name)


def test_rising_scores_move_the_maximum_every_tile():
    B, Nq, Nk, H, D = 1, 200, 700, 1, 64
    q, v, go = randn(B, Nq, H, D), randn(B, Nk, H, D, seed=3), randn(B, Nq, H, D, seed=4)
    q = q.abs()
    k = (torch.arange(Nk, device="cuda")[None, :, None, None] * 0.02).expand(B, Nk, H, D).to(torch.bfloat16)
    k = k.contiguous()
    ref = reference(q, k, v, None, 0.125, go)
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    check(o, ref, "o")
    check(lse, ref, "lse")
    for g, name in zip(hwp.cross_attention_backward(q, k, v, o, lse, go), ("dq", "dk", "dv")):
        check(g, ref, name)


@pytest.mark.parametrize("Nq", [1, 200])
@pytest.mark.parametrize("D", [64, 72])
def test_slices_of_fused_tensors(Nq, D):
    """Queries, keys and values as slices of fused projections, gradients written into slices; a
    head-major output; nothing beside the slices changes."""
    B, Nk, H = 2, 150, 4
    fq, fkv, go = randn(B, Nq, 3, H, D), randn(B, Nk, 2, H, D, seed=2), randn(B, Nq, H, D, seed=3)
    q, k, v = fq[:, :, 1], fkv[:, :, 0], fkv[:, :, 1]
    qc, kc, vc = q.contiguous(), k.contiguous(), v.contiguous()
    want, want_lse = hwp.cross_attention(qc, kc, vc, with_lse=True)
    before = fq.clone()
    o = fq[:, :, 2]  # the output between the queries of the same buffer
    lse = torch.empty_like(want_lse)
    hwp.tok_cross_attention(q, k, v, o, lse)
    assert torch.equal(o, want) and torch.equal(lse, want_lse) and torch.equal(fq[:, :, :2], before[:, :, :2])
    head_major = torch.full((B, H, Nq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    hwp.tok_cross_attention(q, k, v, head_major.transpose(1, 2))
    assert torch.equal(head_major.transpose(1, 2), want)
    grads = hwp.cross_attention_backward(qc, kc, vc, want, want_lse, go)
    gkv = torch.empty_like(fkv)
    gq = torch.full_like(fq, 5.0)
    hwp.tok_cross_attention_backward(q, k, v, o, lse, go, gq[:, :, 0], gkv[:, :, 0], gkv[:, :, 1])
    for a, b in zip((gq[:, :, 0], gkv[:, :, 0], gkv[:, :, 1]), grads):
        assert torch.equal(a, b)
    assert bool((gq[:, :, 1:] == 5.0).all())


@pytest.mark.parametrize("Nq", [1, 300])
def test_head_major_and_batch_inner_layouts(Nq):
    """[B, H, N, D] and [N, B, H, D] memory: the same results as dense tensors."""
    B, Nk, Hq, Hkv, D = 2, 333, 4, 2, 64
    q, k, v, go = (randn(B, n, h, D, seed=s) for n, h, s in ((Nq, Hq, 1), (Nk, Hkv, 2), (Nk, Hkv, 3), (Nq, Hq, 4)))
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    grads = hwp.cross_attention_backward(q, k, v, o, lse, go)
    for perm, back in (((0, 2, 1, 3), (0, 2, 1, 3)), ((1, 0, 2, 3), (1, 0, 2, 3)), ((2, 1, 0, 3), (2, 1, 0, 3))):
        t = [x.permute(perm).contiguous().permute(back) for x in (q, k, v, o, go)]
        o2, lse2 = hwp.cross_attention(*t[:3], with_lse=True)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        for a, b in zip(hwp.cross_attention_backward(*t[:4], lse, t[4]), grads):
            assert torch.equal(a, b)


@pytest.mark.parametrize("Nq", [1, 200])
def test_broadcast_encoder_state(Nq):
    """One encoder state for the whole batch (stride 0), one key head shared by expansion."""
    B, Nk, H, D = 3, 140, 4, 64
    q, go = randn(B, Nq, H, D), randn(B, Nq, H, D, seed=4)
    k, v = randn(1, Nk, 1, D, seed=2).expand(B, Nk, H, D), randn(1, Nk, 1, D, seed=3).expand(B, Nk, H, D)
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    oc, lc = hwp.cross_attention(q, k.contiguous(), v.contiguous(), with_lse=True)
    assert torch.equal(o, oc) and torch.equal(lse, lc)
    got = hwp.cross_attention_backward(q, k, v, o, lse, go)
    for a, b in zip(got, hwp.cross_attention_backward(q, k.contiguous(), v.contiguous(), o, lse, go)):
        assert torch.equal(a, b)


def test_shared_heads_sum_their_gradients():
    """Grouped heads give what separate heads give, summed over the group."""
    B, Nq, Nk, Hq, Hkv, D = 1, 150, 140, 6, 2, 64
    q, k, v, go = randn(B, Nq, Hq, D), randn(B, Nk, Hkv, D, seed=2), randn(B, Nk, Hkv, D, seed=3), randn(B, Nq, Hq, D, seed=4)
    ref = reference(q, k, v, None, D ** -0.5, go)
    sep = reference(q, k.repeat_interleave(3, 2), v.repeat_interleave(3, 2), None, D ** -0.5, go)
    for name in ("dk", "dv"):  # the reference itself
        assert float((sep[name][0].view(B, Nk, Hkv, 3, D).sum(3) - ref[name][0]).abs().max()) < 1e-10
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    for g, name in zip(hwp.cross_attention_backward(q, k, v, o, lse, go), ("dq", "dk", "dv")):
        check(g, ref, name)


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit definition."""
    B, Nq, Nk, H, D = 1, 40, 50, 2, 32
    q, k, v, go = (randn(B, n, H, D, seed=s) for n, s in ((Nq, 1), (Nk, 2), (Nk, 3), (Nq, 4)))
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    grads = hwp.cross_attention_backward(q, k, v, o, lse, go)
    ref = reference(q, k, v, None, D ** -0.5, go)

    def loss(q, k, v):
        s = torch.einsum("bqhd,bkhd->bhqk", q, k) * D ** -0.5
        return (torch.einsum("bhqk,bkhd->bqhd", s.softmax(-1), v) * go.double()).sum()

    x = [t.double() for t in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        d = randn(*x[i].shape, seed=10 + i).double()
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-5 * d, x[i] - 1e-5 * d
        slope = (loss(*up) - loss(*down)) / 2e-5
        tol = (ref[name][1] * d.abs()).sum() + 1e-6 * abs(slope) + 1e-6
        assert abs(float((grads[i].double() * d).sum() - slope)) <= float(tol), name


def test_streams_graphs_and_workspaces():
    """Another stream; a forward and backward captured together and replayed on new inputs beside
    eager calls; two captured calls with a workspace each."""
    B, Nk, H, D = 2, 3000, 4, 64
    k, v = randn(B, Nk, H, D, seed=2), randn(B, Nk, H, D, seed=3)
    for Nq in (1, 150):
        q, go = randn(B, Nq, H, D), randn(B, Nq, H, D, seed=4)
        o, lse = hwp.cross_attention(q, k, v, with_lse=True)
        grads = hwp.cross_attention_backward(q, k, v, o, lse, go)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        o2, lse2 = hwp.cross_attention(q, k, v, with_lse=True, stream=s)
        g2 = hwp.cross_attention_backward(q, k, v, o2, lse2, go, stream=s)
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(grads, g2):
            assert torch.equal(a, b)
        sq = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o3, lse3 = hwp.cross_attention(sq, k, v, with_lse=True)
            o4 = hwp.cross_attention(2 * sq, k, v)
            g3 = hwp.cross_attention_backward(sq, k, v, o3, lse3, go)
        sq.copy_(q)
        graph.replay()
        eager = hwp.cross_attention(2 * q, k, v)
        torch.cuda.synchronize()
        assert torch.equal(o3, o) and torch.equal(lse3, lse) and torch.equal(o4, eager)
        for a, b in zip(grads, g3):
            assert torch.equal(a, b)
        del graph


@pytest.mark.parametrize("Nk", [4000, 40000])
def test_caller_workspace_and_untouched_surroundings(Nk):
    B, Nq, H, D = 1, 2, 2, 64
    q, k, v = randn(B, Nq, H, D), randn(B, Nk, H, D, seed=2), randn(B, Nk, H, D, seed=3)
    need = hwp.cross_attention_workspace_size(B, Nq, Nk, H, H, D)
    assert need > 0 or Nk == 4000  # (a cluster joins the shorter one)
    buf = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((B, Nq + 2, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    hwp.tok_cross_attention(q, k, v, out[:, 1:1 + Nq], workspace=buf[256:256 + need])
    assert torch.equal(out[:, 1:1 + Nq], hwp.cross_attention(q, k, v))
    assert bool((out[:, 0] == 3).all()) and bool((out[:, -1] == 3).all())
    assert bool((buf[:256] == 77).all()) and bool((buf[256 + need:] == 77).all())
    if need:
        with pytest.raises(hwp.TokError) as e:
            hwp.tok_cross_attention(q, k, v, out[:, :Nq], workspace=buf[256:256 + need - 16])
        assert e.value.status == hwp.TOK_ERR_SHAPE


@pytest.mark.parametrize("B,Nq,Nk,Hq,Hkv,D", [(4, 1, 3000, 8, 2, 128), (1, 2437, 1500, 16, 16, 128), (2, 1300, 900, 16, 4, 64)])
def test_two_streams_at_once(B, Nq, Nk, Hq, Hkv, D):
    """Calls that run beside each other on two streams, each with partial results in a workspace of its own."""
    data = [[randn(B, n, h, D, seed=10 * i + s) for s, (n, h) in enumerate(((Nq, Hq), (Nk, Hkv), (Nk, Hkv), (Nq, Hq)))]
            for i in range(2)]
    def call(q, k, v, go):
        o, lse = hwp.cross_attention(q, k, v, with_lse=True)
        return (o, lse) + tuple(hwp.cross_attention_backward(q, k, v, o, lse, go))
    want = [call(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(*data[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, run))
    hwp.tok_check_device()


def test_empty_calls():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert hwp.cross_attention(e(0, 3, 2, 64), e(0, 5, 2, 64), e(0, 5, 2, 64)).numel() == 0
    assert hwp.cross_attention(e(2, 0, 2, 64), e(2, 5, 2, 64), e(2, 5, 2, 64)).numel() == 0
    o, lse = hwp.cross_attention(e(2, 0, 2, 64), e(2, 5, 2, 64), e(2, 5, 2, 64), with_lse=True)
    dq, dk, dv = hwp.cross_attention_backward(e(2, 0, 2, 64), e(2, 5, 2, 64), e(2, 5, 2, 64), o, lse, e(2, 0, 2, 64))
    assert dq.numel() == 0 and bool((dk == 0).all()) and bool((dv == 0).all())


def test_a_step_of_a_code_model():
    """Positions, attention of grid tokens over a conditioning frame's tokens, logits, a drawn code,
    its latent: the operators as one run, each against its own definition."""
    t, h, w, Hq, Hkv, D = 1, 6, 10, 4, 2, 64
    dims, sizes = (24, 20, 20), (4, 8, 12)
    table = hwp.rope_table(sizes, dims)
    q, k, v = randn(2, t, h, w, Hq, D), randn(2, 2, h, w, Hkv, D, seed=2), randn(2, 2, h, w, Hkv, D, seed=3)
    qr = hwp.rope_grid(q, table, sizes, dims, origin=(2, 0, 0)).view(2, -1, Hq, D)
    kr = hwp.rope_grid(k, table, sizes, dims).view(2, -1, Hkv, D)
    vv = v.view(2, -1, Hkv, D)
    lens = torch.tensor([120, 60], dtype=torch.int32, device="cuda")
    o, lse = hwp.cross_attention(qr, kr, vv, lens, with_lse=True)
    go = randn(2, h * w, Hq, D, seed=5)
    ref = reference(qr, kr, vv, lens, D ** -0.5, go)
    check(o, ref, "o")
    dq, dk, _ = hwp.cross_attention_backward(qr, kr, vv, o, lse, go, lens)
    check(dq, ref, "dq")
    gq = hwp.rope_grid_adjoint(dq.view_as(q), table, sizes, dims, origin=(2, 0, 0))
    back = hwp.rope_grid(gq, table, sizes, dims, origin=(2, 0, 0)).view_as(dq)  # two roundings, rotated once
    pair = dq.double().abs() + dq.double().abs().roll(D // 2, -1)
    assert bool(((back.double() - dq.double()).abs() <= (2 * RB + 8 * U) * 2 * pair).all())
    wl = randn(Hq * D, hwp.FSQ_CODEBOOK, seed=6, spread=0.2)
    logits = o.reshape(2 * h * w, Hq * D) @ wl
    u = torch.rand(2 * h * w, generator=torch.Generator(device="cuda").manual_seed(7), device="cuda")
    idx = hwp.sample_codes(logits, u, temperature=0.9, top_k=200, top_p=0.95)
    top = logits.float().topk(200, dim=1).values[:, -1]
    assert bool((logits.float().gather(1, idx.long()[:, None])[:, 0] >= top).all())
    latent = hwp.fsq_decode(idx.view(2, 1, h, w), torch.randn(6, 16, device="cuda"))
    assert latent.shape == (2, 16, 1, h, w) and bool(latent.isfinite().all())


@pytest.mark.parametrize("Nq,Nk,H,D,dead", [(3, 400, 2, 64, 130), (2, 6000, 2, 128, 3000), (300, 400, 2, 64, 130),
                                            (300, 400, 2, 128, 256), (1200, 2600, 5, 128, 1900), (260, 700, 3, 64, 700)])
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("level", [-150.0, 0.0, 90.0])
def test_keys_masked_through_a_channel(Nq, Nk, H, D, dead, low, level):
    """Keys ruled out by a channel of their own (1 in the queries, -inf or the lowest number in the keys): whole
    tiles of them before keys whose scores lie at any level."""
    q, k, v = (randn(1, n, H, D, seed=s, spread=f) for n, s, f in ((Nq, 1, 1.0), (Nk, 2, 0.3), (Nk, 3, 1.0)))
    q[..., 0], q[..., 1] = 1.0, 1.0
    k[..., 0], k[..., 1] = 0.0, level
    live = k[:, dead:].contiguous(), v[:, dead:].contiguous()
    k[:, :dead, :, 0] = low
    o, lse = hwp.cross_attention(q, k, v, scale=1.0, with_lse=True)
    if dead == Nk:
        if low == -math.inf:
            assert bool((o == 0).all()) and bool((lse == -math.inf).all())
        return
    ref = reference(q, *live, None, 1.0)
    check(o, ref, "o")
    check(lse, ref, "lse")


@pytest.mark.parametrize("B,Nq,Nk,H,D", [(1, 3, 90, 2, 64), (1, 2, 6000, 2, 128), (1, 300, 300, 2, 64),
                                         (1, 1200, 2600, 5, 128)])
def test_nan_in_live_places_shows(B, Nq, Nk, H, D):
    """A query, or a key within the length, of NaN: what the formula makes NaN is NaN, the statistics as well, and
    nothing else changes."""
    q, k, v, go = (randn(B, n, H, D, seed=s) for n, s in ((Nq, 1), (Nk, 2), (Nk, 3), (Nq, 4)))
    clean, clean_lse = hwp.cross_attention(q, k, v, with_lse=True)
    row = Nq // 2
    q[0, row, 1] = math.nan
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    assert bool(o[0, row, 1].isnan().all()) and bool(lse[0, 1, row].isnan())
    o[0, row, 1], lse[0, 1, row] = clean[0, row, 1], clean_lse[0, 1, row]
    assert torch.equal(o, clean) and torch.equal(lse, clean_lse)
    q[0, row, 1] = 1.0
    k[0, Nk - 2, 0, 5] = math.nan
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    assert bool(o[:, :, 0].isnan().all()) and bool(lse[:, 0].isnan().all())
    assert bool(o[:, :, 1].isfinite().all()) and bool(lse[:, 1].isfinite().all())
    dq, dk, dv = hwp.cross_attention_backward(q, k, v, o, lse, go)
    for g in (dq, dk, dv):
        assert bool(g[:, :, 0].isnan().all()) and bool(g[:, :, 1].isfinite().all())


def test_gradients_ask_for_the_statistics():
    x = randn(1, 2, 2, 64)
    with pytest.raises(ValueError, match="lse"):
        hwp.cross_attention_backward(x, x, x, x, None, x)


def test_no_queries_and_very_many_key_heads():
    """Gradients of 134 million rows of keys and values without a query (69 GB): zeros."""
    B, H, D = 8192, 16400, 128
    e = torch.empty(B, 0, H, D, dtype=torch.bfloat16, device="cuda")
    k = randn(1, 1, 1, D).expand(B, 1, H, D)
    dk, dv = (torch.full((B, 1, H, D), 1.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hwp.tok_cross_attention_backward(e, k, k, e, torch.empty(B, H, 0, device="cuda"), e, e, dk, dv)
    for g in (dk, dv):
        bits = g.view(torch.int32)
        assert int(bits.max()) == 0 and int(bits.min()) == 0
    del dk, dv, g, bits
    torch.cuda.empty_cache()


@pytest.mark.parametrize("case", [  # few query rows in more than one tile of 16, keys in more than one split
    (1, 40, 3000, 2, 2, 128, None), (2, 12, 2000, 12, 4, 80, "ragged"), (1, 17, 4000, 1, 1, 64, None),
    (3, 11, 1500, 8, 2, 72, "wild"),
    # on both sides of the border between the two kernels: 48 and 49, 64 query rows of a key head
    (2, 12, 1500, 8, 2, 128, "ragged"), (1, 48, 1000, 2, 2, 64, None), (1, 49, 1000, 2, 2, 64, None),
    (2, 16, 1500, 8, 2, 128, "ragged"), (2, 7, 900, 14, 2, 96, "empty")])
def test_rows_by_tiles_and_splits(case):
    test_forward(case)
    test_backward(case)


@pytest.mark.parametrize("B,Nq,Nk,Hq,Hkv,D", [(1, 2, 4000, 2, 2, 64), (1, 2, 40000, 2, 2, 64), (1, 2437, 1500, 16, 16, 128)])
def test_workspaces_are_taken_and_checked(B, Nq, Nk, Hq, Hkv, D):
    """Split calls in a workspace of the caller's, with nothing to spare; one byte less is refused."""
    q, k, v, go = randn(B, Nq, Hq, D), randn(B, Nk, Hkv, D, seed=2), randn(B, Nk, Hkv, D, seed=3), randn(B, Nq, Hq, D, seed=4)
    o, lse = hwp.cross_attention(q, k, v, with_lse=True)
    grads = hwp.cross_attention_backward(q, k, v, o, lse, go)
    dims = B, Nq, Nk, Hq, Hkv, D
    need, back = hwp.cross_attention_workspace_size(*dims), hwp.cross_attention_backward_workspace_size(*dims)
    assert need > 0 and back > 0
    buf = torch.full((max(need, back) + 512,), 77, dtype=torch.uint8, device="cuda")
    for n, call, want in (
            (need, lambda ws: (hwp.tok_cross_attention(q, k, v, torch.empty_like(q), workspace=ws),), (o,)),
            (back, lambda ws: hwp.tok_cross_attention_backward(q, k, v, o, lse, go, torch.empty_like(q), torch.empty_like(k),
                                                               torch.empty_like(v), workspace=ws), grads)):
        buf.fill_(77)
        assert all(torch.equal(a, b) for a, b in zip(call(buf[256:256 + n]), want))
        assert bool((buf[:256] == 77).all()) and bool((buf[256 + n:] == 77).all())
        with pytest.raises(hwp.TokError) as e:
            call(buf[256:256 + n - 1])
        assert e.value.status == hwp.TOK_ERR_SHAPE


@pytest.mark.parametrize("Nq,Nk,Hq,Hkv,D,dead", [(3, 100, 2, 2, 64, 40), (1, 400, 6, 2, 128, 130), (300, 400, 2, 2, 64, 130),
                                                 (256, 400, 2, 1, 128, 256), (1201, 2600, 4, 2, 128, 1900)])
@pytest.mark.parametrize("low", [-math.inf, torch.finfo(torch.bfloat16).min])
def test_gradients_of_keys_masked_through_a_channel(Nq, Nk, Hq, Hkv, D, dead, low):
    """Keys ruled out by a channel of their own get no gradient, whether or not the queries fill their tiles; the
    others get what they get alone.  (That channel of grad_q is 0 times -inf: NaN by the formula.)"""
    q, k, v, go = (randn(1, n, h, D, seed=s, spread=f)
                   for n, h, s, f in ((Nq, Hq, 1, 1.0), (Nk, Hkv, 2, 0.3), (Nk, Hkv, 3, 1.0), (Nq, Hq, 4, 1.0)))
    q[..., 0], k[..., 0] = 1.0, 0.0
    ref = reference(q, k[:, dead:].contiguous(), v[:, dead:].contiguous(), None, 1.0, go)
    k[:, :dead, :, 0] = low
    o, lse = hwp.cross_attention(q, k, v, scale=1.0, with_lse=True)
    dq, dk, dv = hwp.cross_attention_backward(q, k, v, o, lse, go, scale=1.0)
    assert bool((dk[:, :dead] == 0).all()) and bool((dv[:, :dead] == 0).all())
    check(dk[:, dead:], ref, "dk")
    check(dv[:, dead:], ref, "dv")
    if low == -math.inf:
        assert bool(dq[..., 0].isnan().all())
        dq[..., 0] = ref["dq"][0][..., 0].to(dq.dtype)
    check(dq, ref, "dq")
