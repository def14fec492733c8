"""Drawing codes against a plain implementation in 64 bits (numpy, row by row).

Indices have to be equal.  The kernel's weights are within 2^-45 of the definition's (relative
to the largest), so a draw differs only if u lies within V * 2^-45 < 2^-27 of a border: the
reference says how near the nearest border is, and rows nearer than 2^-26 are left out (none
of the seeded rows is).  logprob: z and ln(total) are taken in 64 bits and rounded to fp32
once, 2^-24 relative; the weights' 2^-45 each move ln(total) by at most V * 2^-45 < 2^-27.
"""
import math

import numpy as np
import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

V0 = hwp.FSQ_CODEBOOK


def reference(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row -> (index, ln probability, distance of u to the nearest border or filter limit)."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    temperature, top_p, min_p, u = (float(np.float32(v)) for v in (temperature, top_p, min_p, u))
    if np.all(x == -np.inf):
        return -1, -math.inf, 1.0
    order = np.argsort(-x, kind="stable")
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    order = order[x[order] > -np.inf]
    if top_k > 0:
        order = order[:top_k]
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(x[order] == x[order[0]], 0.0, (x[order] - x[order[0]]) / temperature))
    near = 1.0
    if top_p < 1:
        before = np.cumsum(w) - w
        total = w.sum()
        if top_p > 0:
            near = min(near, float(np.min(np.abs(before - top_p * total)[w > 0])) / total) if len(set(w)) > 1 else near
        keep = before < top_p * total
        keep[0] = True
        order, w = order[keep], w[keep]
    keep = w >= min(max(min_p, 0.0), 1.0)
    order, w = order[keep], w[keep]
    by = np.argsort(order)
    order, w = order[by], w[by]
    c = np.cumsum(w)
    near = min(near, float(np.min(np.abs(c[:-1] - u * c[-1]))) / c[-1]) if len(c) > 1 else near
    n = int(np.searchsorted(c, min(max(u, 0.0), 1.0) * c[-1], side="right"))
    n = min(n, int(np.nonzero(w > 2.0 ** -45)[0][-1]))
    return int(order[n]), math.log(w[n] / c[-1]), near


def compare(logits, u, label="", **settings):
    """Every row of logits [R, V] against the reference."""
    dev = {k: (torch.as_tensor(v, device="cuda") if isinstance(v, np.ndarray) else v) for k, v in settings.items()}
    idx, lp = hwp.sample_codes(logits, u, with_logprob=True, **dev)
    x, uu = logits.float().cpu().numpy(), u.cpu().numpy()
    skipped = 0
    for r in range(len(uu)):
        row = {k: (v[r] if isinstance(v, np.ndarray) else v) for k, v in settings.items()}
        want, want_lp, near = reference(x[r], uu[r], **row)
        if near < 2.0 ** -26:
            skipped += 1
            continue
        assert int(idx[r]) == want, f"{label} row {r}: drew {int(idx[r])}, expected {want} ({row})"
        if math.isinf(want_lp):
            assert float(lp[r]) == want_lp
        else:
            assert abs(float(lp[r]) - want_lp) <= 2.0 ** -24 * abs(want_lp) + 2.0 ** -26, f"{label} row {r}"
    assert skipped <= len(uu) // 4
    return idx


def data(R, V, spread=2.0, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(R, V, generator=g, device="cuda") * spread).to(dtype)
    return x, torch.rand(R, generator=g, device="cuda")


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.1),
            dict(temperature=0.8, top_k=100, top_p=0.95, min_p=0.02), dict(top_k=1), dict(temperature=0.0),
            dict(top_p=0.0), dict(top_p=1e-6, top_k=1000), dict(temperature=1.3, top_k=3000, top_p=0.99),
            dict(min_p=1.0), dict(min_p=7.0), dict(temperature=100.0, top_p=0.5), dict(temperature=0.01, top_p=0.5)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", SETTINGS)
@pytest.mark.parametrize("R,V", [(3, V0), (40, 4097), (150, 257)])
def test_filters(R, V, settings, dtype):
    x, u = data(R, V, dtype=dtype)
    compare(x, u, **settings)


@pytest.mark.parametrize("V", [1, 2, 31, 255, 256, 1025, 8191, 65537, 1 << 18])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabulary_sizes(V, dtype):
    x, u = data(2, V, dtype=dtype, seed=V)
    compare(x, u, top_k=max(1, V // 3), top_p=0.8)
    compare(x, u)


@pytest.mark.parametrize("R", [1, 20, 40, 80, 200, 500])
def test_rows_of_every_cluster_size(R):
    x, u = data(R, 12345, dtype=torch.bfloat16, seed=R)
    compare(x, u, top_k=77, top_p=0.9)


def test_settings_per_row():
    R = 24
    x, u = data(R, 5000, seed=5)
    rng = np.random.RandomState(0)
    compare(x, u, temperature=np.float32([0.0, 1.0, 0.5, 2.0] * 6),
            top_k=rng.choice([0, -3, 1, 5, 400, 5000, 9999], R).astype(np.int32),
            top_p=rng.choice([1.0, 0.3, 0.9, 0.0, 1.5], R).astype(np.float32),
            min_p=rng.choice([0.0, 0.05, -1.0], R).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", [dict(top_k=37), dict(top_p=0.37), dict(top_k=3000, top_p=0.7), dict(top_k=1),
                                      dict(temperature=0.0), dict()])
def test_ties(settings, dtype):
    """Few different values, each thousands of times: the lower index first."""
    V = 30001
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 3, (9, V), generator=g, device="cuda").to(dtype)
    x[0] = 1.5
    x[1] = torch.where(torch.arange(V, device="cuda") == 17, 2.0, -1.0)
    x[2, ::2], x[2, 1::2] = 0.0, -0.0
    u = torch.linspace(0, 0.999, 9, device="cuda") + 1e-4
    compare(x, u.clamp(max=0.9999), "ties", **settings)


def test_narrow_and_far_values():
    """Clusters that one histogram bin holds, beside values far off."""
    V = 20000
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(8, V, generator=g, device="cuda") * 1e-3
    x[0:2] += 20.0
    x[2:4, 0] = 15.0              # one token above a narrow cluster
    x[4, 10:] = -1e9              # masked with a large finite value
    x[5, 10:] = torch.finfo(torch.float32).min
    x[6, : V // 2] -= 25.0
    u = torch.rand(8, generator=g, device="cuda")
    for s in (dict(top_k=5000), dict(top_p=0.5), dict(top_k=9000, top_p=0.9), dict(top_k=9), dict(temperature=0.01)):
        compare(x, u, "narrow", **s)


def test_infinities_nan_and_empty_rows():
    V = 3000
    x, u = data(8, V, seed=3)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 5:] = -math.inf
    x[3, ::3] = math.nan
    x[4, 100] = x[4, 7] = math.inf
    x[5, 1:] = math.nan
    x[6, : V - 1] = torch.finfo(torch.float32).min
    x[6, V - 1] = torch.finfo(torch.float32).min
    for s in (dict(), dict(top_k=10, top_p=0.9), dict(top_p=0.5, temperature=2.0), dict(temperature=0.0)):
        idx = compare(x, u, "special", **s)
        assert idx[:2].tolist() == [-1, -1]
    compare(x, u, "infinite temperature", temperature=3.4e38, top_k=2000)


def test_draws_at_the_ends():
    x, _ = data(4, 1000, seed=4)
    u = torch.tensor([0.0, 1.0, 2.0, -1.0], device="cuda")
    idx = hwp.sample_codes(x, u)
    assert idx.tolist() == [0, 999, 999, 0]
    x[:, 990:] = -math.inf
    x[:, :3] = -math.inf
    assert hwp.sample_codes(x, u).tolist() == [3, 989, 989, 3]
    assert hwp.sample_codes(x, torch.full_like(u, math.nan)).tolist() == [3] * 4


def test_strided_rows_and_addresses():
    for off in (0, 1, 3):
        buf, u = data(1, off + 6 * 1100, dtype=torch.bfloat16, seed=6)
        x = buf[0, off:].view(6, 1100)[:, 50:1050]
        before = buf.clone()
        compare(x, data(6, 1)[1], top_k=40)
        assert torch.equal(buf, before)
    x, u = data(1, 700)
    same = x.expand(5, 700)
    assert hwp.sample_codes(same, u.expand(5).contiguous()).unique().numel() == 1


def test_distribution():
    """20,000 draws of one row against its probabilities: a chi-square of 19 degrees beyond 63 has
    a chance of 1e-6."""
    p = torch.rand(20, generator=torch.Generator().manual_seed(7)) + 0.1
    x = p.log().cuda().expand(20000, 20)
    u = torch.rand(20000, generator=torch.Generator().manual_seed(8)).cuda()
    n = torch.bincount(hwp.sample_codes(x, u).long(), minlength=20).double().cpu()
    want = (p / p.sum()).double() * 20000
    assert float(((n - want) ** 2 / want).sum()) < 63


def test_graph_stream_repeat_and_empty():
    x, u = data(5, V0, dtype=torch.bfloat16, seed=9)
    want = hwp.sample_codes(x, u, top_k=300, top_p=0.9)
    for _ in range(5):
        assert torch.equal(hwp.sample_codes(x, u, top_k=300, top_p=0.9), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = hwp.sample_codes(x, u, top_k=300, top_p=0.9, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    static, idx = torch.zeros_like(x), torch.empty(5, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hwp.tok_sample_codes(static, u, idx, top_k=300, top_p=0.9)
    static.copy_(x)
    g.replay()
    assert torch.equal(idx, want)
    assert hwp.sample_codes(torch.empty(0, 10, device="cuda"), torch.empty(0, device="cuda")).numel() == 0
    assert hwp.sample_codes(x[0], u[0]).shape == ()


def test_feeds_fsq_decode():
    x, u = data(12, V0, seed=10)
    x[3] = -math.inf
    idx = hwp.sample_codes(x, u, top_p=0.9).view(1, 3, 4)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = hwp.fsq_decode(idx, torch.randn(6, 16, device="cuda"), bad)
    assert int(bad) == 1 and out.shape == (1, 16, 3, 4)
    assert out[0, :, 0, 3].isnan().all() and out.isnan().sum() == 16


@pytest.mark.parametrize("R", [1, 9, 400])
@pytest.mark.parametrize("V", [V0, 5000])
def test_samples_that_mislead(R, V):
    """Rows whose sampled part says nothing about the rest: all of it ruled out, or infinite, or the
    largest tokens all elsewhere; and rows with few tokens left."""
    x, u = data(R, V, seed=11)
    step = torch.arange(V, device="cuda")
    x[0, step % 2048 < 256] = -math.inf
    compare(x[:1], u[:1], top_k=100, top_p=0.9)
    x[0] = torch.where(step % 2048 < 256, -5.0, 5.0) + 0.1 * x[0].nan_to_num(0.0, 0.0, 0.0)
    compare(x[:1], u[:1], top_k=300)
    x[0, V // 2] = math.inf
    x[0, 3] = math.inf
    compare(x[:1], u[:1], top_k=300, top_p=0.9)
    x[0] = -math.inf
    x[0, V - 1] = x[0, V // 3] = 1.0
    idx = compare(x[:3], u[:3], top_k=50, top_p=0.4)
    compare(x[:3], u[:3], top_p=0.4)
    compare(x[:3], u[:3], top_k=2000, top_p=0.4)
    if R > 3:
        assert torch.equal(hwp.sample_codes(x, u, top_k=50, top_p=0.4)[:3], idx[:3])


def test_two_streams_at_once():
    """Calls on two streams at the same time, with settings per row, give what each gives alone."""
    a, b = data(40, V0, dtype=torch.bfloat16, seed=12), data(300, 9000, seed=13)
    k = torch.randint(1, 900, (300,), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    want = hwp.sample_codes(*a, top_p=0.8), hwp.sample_codes(*b, top_k=k)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x, y = hwp.sample_codes(*a, top_p=0.8, stream=s1), hwp.sample_codes(*b, top_k=k, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


def drawn(x, u, temperature, min_p, idx, lp, label):
    """One draw without a rank limit against the running sum in 64 bits.  Weights are off by at most half a
    unit of 2^-44 and 2^-44 of themselves (the exponential), so the sums before and through the drawn token are
    off by at most V 2^-45 + 2^-44 total, and so is u times the total: a slack of twice both; a token below half a unit
    has no weight at all."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    t, floor = float(np.float32(temperature)), float(np.float32(min_p))
    w = np.exp((x - x.max()) / t)
    w[w < floor] = 0.0
    c = np.cumsum(w)
    slack = 2 * (len(x) * 2.0 ** -45 + 2.0 ** -44 * c[-1])
    assert 0 <= idx < len(x), f"{label}: index {idx}"
    assert w[idx] > 2.0 ** -45 * (1 - 2.0 ** -40), f"{label}: drew {idx}, whose weight is {w[idx]}"
    at = min(max(float(u), 0.0), 1.0) * c[-1]
    assert c[idx] - w[idx] - slack <= at <= c[idx] + slack, f"{label}: drew {idx}"
    want = math.log(w[idx] / c[-1])
    assert abs(lp - want) <= 2.0 ** -24 * abs(want) + 2.0 ** -26, f"{label}: {lp}, expected {want}"


COLD = [1e-4, 1e-5, 1e-6, 1e-7, 1e-8, 1e-12, 1e-38, 1e-45]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [V0, 4097])
@pytest.mark.parametrize("R", [4, 40, 320])
@pytest.mark.parametrize("min_p", [0.0, 0.3])
def test_temperatures_next_to_zero(R, V, dtype, min_p):
    """Temperatures at which a token's reach is below a step of the largest logit: tokens far below it, -inf
    and NaN, in front, behind and between, have no weight, whatever u is."""
    for top in (1.0, 9.0, 24.0, 100.0, 200.0, 1000.0):
        x, _ = data(R, V, dtype=torch.float32, seed=int(top))
        x = top - 0.02 * top - 0.1 * x.abs()
        x[:, : V // 8] = -math.inf
        x[:, V - V // 8:] = math.nan
        x[1::2, V - V // 8:] = -math.inf
        x[:, V // 2: V // 2 + 40: 8] = top
        x[2::3, V // 3] = top * (1 - 2.0 ** -23)  # one step below
        x = x.to(dtype)
        temperature = torch.tensor([COLD[r % len(COLD)] for r in range(R)], device="cuda")
        u = torch.tensor([(0.0, 0.5, 1 - 2.0 ** -24, 1.0, 0.3)[r // len(COLD) % 5] if R > 4 else (0.0, 0.5, 1.0, 0.3)[r]
                          for r in range(R)], device="cuda")
        if R == 4:
            temperature = temperature.roll(int(top) % 4) * 1e-2
        idx = torch.full((R,), -7, dtype=torch.int32, device="cuda")
        lp = torch.full((R,), 7.0, device="cuda")
        hwp.tok_sample_codes(x, u, idx, lp, temperature=temperature, min_p=min_p)
        xs, i, p, t, us = x.float().cpu().numpy(), idx.tolist(), lp.tolist(), temperature.tolist(), u.tolist()
        for r in range(R if R < 320 else 120):
            drawn(xs[r], us[r], t[r], min_p, i[r], p[r], f"top {top} row {r} T {t[r]} u {us[r]}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R", [3, 60, 320])
def test_cold_nucleus_of_equal_values(R, dtype):
    """Many equal largest values under top_p: the tokens below them do not count in its total."""
    V, n = 600, 401
    g = torch.Generator(device="cuda").manual_seed(14)
    for top in (1.0, 24.0, 1000.0):
        x = torch.full((R, V), top, device="cuda")
        for r in range(R):
            x[r, torch.randperm(V, generator=g, device="cuda")[: V - n]] = (0.5 * top, -math.inf, math.nan)[r % 3]
        u = torch.rand(R, generator=g, device="cuda")
        for t in (1e-6, 1e-8, 1e-38):
            for top_p in (0.3, 0.5, 0.6):
                for s in (dict(), dict(min_p=0.2)):
                    compare(x.to(dtype)[:60], u[:60], f"top {top}", temperature=t, top_p=top_p, **s)
                    if R > 60:
                        want = hwp.sample_codes(x[:60].to(dtype), u[:60].contiguous(), temperature=t, top_p=top_p, **s)
                        got = hwp.sample_codes(x.to(dtype), u, temperature=t, top_p=top_p, **s)
                        assert torch.equal(got[:60], want)


def check_some(x, u, rows, label="", **settings):
    """One call over all rows; `rows` of them against the reference."""
    dev = {k: (torch.as_tensor(v, device="cuda") if isinstance(v, np.ndarray) else v) for k, v in settings.items()}
    idx, lp = hwp.sample_codes(x, u, with_logprob=True, **dev)
    sub, uu, idx, lp = x[rows].float().cpu().numpy(), u[rows].tolist(), idx[rows].tolist(), lp[rows].tolist()
    skipped = 0
    for i, r in enumerate(rows):
        row = {k: (v[r] if isinstance(v, np.ndarray) else v) for k, v in settings.items()}
        want, want_lp, near = reference(sub[i], uu[i], **row)
        if near < 2.0 ** -26:
            skipped += 1
            continue
        assert idx[i] == want, f"{label} row {r}: drew {idx[i]}, expected {want} ({row})"
        if math.isinf(want_lp):
            assert lp[i] == want_lp
        else:
            assert abs(lp[i] - want_lp) <= 2.0 ** -24 * abs(want_lp) + 2.0 ** -26, f"{label} row {r}"
    assert skipped <= len(rows) // 4


MANY = 320  # rows: more than two to an SM, which take blocks of 256 threads


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", SETTINGS + [dict(top_k=500), dict(top_k=900, top_p=0.9), dict(top_k=1025)])
@pytest.mark.parametrize("V", [V0, 4097, 257])
def test_filters_with_many_rows(V, settings, dtype):
    x, u = data(MANY, V, dtype=dtype, seed=15)
    check_some(x, u, [0, 1, 2, 147, 148, 149, 295, 296, 297, 318, 319], **settings)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", [dict(top_k=37), dict(top_p=0.37), dict(top_k=3000, top_p=0.7), dict(top_k=1),
                                      dict(temperature=0.0), dict(), dict(top_k=700)])
def test_ties_narrow_and_special_with_many_rows(settings, dtype):
    V = 9001
    x, _ = data(MANY, V, dtype=torch.float32, seed=16)
    g = torch.Generator(device="cuda").manual_seed(17)
    x[:9] = torch.randint(0, 3, (9, V), generator=g, device="cuda").float()
    x[1] = 1.5
    x[2] = torch.where(torch.arange(V, device="cuda") == 17, 2.0, -1.0)
    x[3, ::2], x[3, 1::2] = 0.0, -0.0
    x[10:14] = 20.0 + 1e-3 * x[10:14]
    x[12:14, 0] = 35.0
    x[14, 10:] = -1e9
    x[15, 10:] = torch.finfo(torch.float32).min
    x[16, : V // 2] -= 25.0
    x[300] = -math.inf
    x[301] = math.nan
    x[302, 5:] = -math.inf
    x[303, ::3] = math.nan
    x[304, 100] = x[304, 7] = math.inf
    x[305, 1:] = math.nan
    u = torch.linspace(0.0101, 0.9897, MANY, device="cuda")
    check_some(x.to(dtype), u, list(range(20)) + list(range(298, 308)), "special", **settings)


def test_settings_per_row_with_many_rows():
    x, u = data(MANY, 5000, seed=18)
    rng = np.random.RandomState(1)
    check_some(x, u, list(range(0, MANY, 8)), temperature=np.float32([0.0, 1.0, 0.5, 2.0, 0.8] * 64),
               top_k=rng.choice([0, -3, 1, 5, 400, 900, 5000, 9999], MANY).astype(np.int32),
               top_p=rng.choice([1.0, 0.3, 0.9, 0.0, 1.5], MANY).astype(np.float32),
               min_p=rng.choice([0.0, 0.05, -1.0], MANY).astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("settings", [dict(top_k=50), dict(top_k=2000), dict(top_p=0.7), dict(top_k=3, top_p=0.9),
                                      dict(top_k=2000, top_p=0.45, min_p=0.1)])
@pytest.mark.parametrize("R", [24, 320])
def test_cold_draws_under_filters(R, settings, dtype):
    """Five equal largest tokens far above the rest, at temperatures next to zero."""
    V = 5000
    g = torch.Generator(device="cuda").manual_seed(19)
    for top in (1.0, 24.0, 1000.0):
        x = 0.5 * top - torch.rand(R, V, generator=g, device="cuda")
        x[:, 100::1000] = top
        x[:, :50] = -math.inf
        x[:, V - 50:] = math.nan
        u = torch.rand(R, generator=g, device="cuda")
        check_some(x.to(dtype), u, list(range(24)), f"top {top}",
                   temperature=np.float32([COLD[r % len(COLD)] for r in range(R)]), **settings)


@pytest.mark.parametrize("R", [2, 400])
def test_one_value_everywhere(R):
    """The longest row, all equal: every token in one bin of the histograms, whose 32-bit sums wrap."""
    V = 1 << 18
    x = torch.full((R, V), -3.0, dtype=torch.bfloat16, device="cuda")
    u = (torch.arange(R, device="cuda") + 0.37) / R
    for top_p in (1.0, 0.25 + 2.0 ** -12, 1e-6, 0.999):
        n = V if top_p >= 1 else math.ceil(float(np.float32(top_p)) * V)
        idx, lp = hwp.sample_codes(x, u, top_p=top_p, with_logprob=True)
        assert idx.tolist() == [int(float(np.float32(t)) * n) for t in u.tolist()], top_p
        assert float((lp + math.log(n)).abs().max()) <= 2.0 ** -24 * math.log(n) + 2.0 ** -26
