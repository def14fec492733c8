"""Attention of new tokens over pages against a 64-bit implementation.

Tolerance, from the arithmetic (u = 2^-24; bf16 rounds by at most 2^-8 of the value):
  scores     products of bf16 are exact in fp32, D of them accumulate, so a score (times
             log2 e) is within S = 2 (D + 4) u max sum|q k| |scale| log2 e of the exact one
             (a factor 2 for the accumulator's internal rounding).
  weights    p = 2^(s - m) / l is within a relative E = 2 S + 2^-21 of the exact one (the
             2-ulp power, the sum and the quotient).  As an operand it is rounded once, 2^-8.
  underflow  the power gives 0 for results below 2^-126, so a weight is also off by up to 2^-126 (TINY).
  o          sum p |v| (2^-8 + E + 2 n u) over n keys, then one rounding of o.
  lse        E + 4 u |lse| + 2 n u.
"""
import math
import random

import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

U, RB = 2.0 ** -24, 2.0 ** -8 * (1 + 2.0 ** -7)
L2E = 1.4426950408889634
TINY = 2.0 ** -126
NAN, INF = float("nan"), float("inf")


def randn(*shape, seed=1, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * spread).to(torch.bfloat16)


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(lens, page, Hkv, D, M=None, seed=1, spare=3):
    """Pages for streams of these lengths, in any order in the pool: (k_pages, v_pages, table)."""
    rng = random.Random(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    M = max(need + [1]) if M is None else M
    order = rng.sample(range(sum(need) + spare), sum(need))
    table = [[order.pop() for _ in range(min(n, M))] + [-1] * (M - n) for n in need]
    pool = randn(sum(need) + spare, 2, page, Hkv, D, seed=seed)
    return pool[:, 0], pool[:, 1], dev(table).view(len(lens), M)


def reference(q, kp, vp, table, k_lens, q_lens=None, scale=None):
    """float64 (o, its tolerance, lse, its tolerance), over the keys that each query sees."""
    B, Nq, Hq, D = q.shape
    page, Hkv = kp.shape[1:3]
    G, scale = Hq // Hkv, D ** -0.5 if scale is None else scale
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    o, to, lse, tl = z(B, Nq, Hq, D), z(B, Nq, Hq, D), z(B, Hq, Nq) - math.inf, z(B, Hq, Nq)
    for b in range(B):
        n = max(0, min(int(k_lens[b]), table.shape[1] * page))
        m = Nq if q_lens is None else max(0, min(Nq, int(q_lens[b])))
        mine = table[b, : -(-n // page)].long()
        for i in range(m):
            see = n - m + i + 1
            if see <= 0:
                continue
            for h in range(Hq):
                kk = kp[mine, :, h // G].reshape(-1, D)[:see].double()
                vv = vp[mine, :, h // G].reshape(-1, D)[:see].double()
                qq = q[b, i, h].double()
                s = scale * kk @ qq
                S = 2 * (D + 4) * U * abs(scale) * L2E * float((kk.abs() @ qq.abs()).max())
                E = 2 * S + 2.0 ** -21
                lse[b, h, i] = torch.logsumexp(s, 0)
                tl[b, h, i] = E + 4 * U * lse[b, h, i].abs() + 2 * see * U
                p = (s - lse[b, h, i]).exp()
                o[b, i, h] = p @ vv
                to[b, i, h] = (p @ vv.abs()) * (RB + E + 2 * see * U) + RB * o[b, i, h].abs() + TINY * vv.abs().sum(0)
    return o, to, lse, tl


def check(got, want, tol, name):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), f"{name}: infinities differ"
    err, tol = (got - want).abs()[fine], tol[fine]
    assert bool((err <= tol + 1e-37).all()), \
        f"{name}: {int((err > tol).sum())} of {err.numel()} beyond the bound, worst {float((err / (tol + 1e-37)).max()):.3g} times it"


def both(q, kp, vp, table, k_lens, q_lens=None, scale=None):
    want = reference(q, kp, vp, table, k_lens, q_lens, scale)
    o, lse = hwp.paged_attention(q, kp, vp, table, k_lens, q_lens, scale, with_lse=True)
    check(o, want[0], want[1], "o")
    check(lse, want[2], want[3], "lse")
    assert torch.equal(hwp.paged_attention(q, kp, vp, table, k_lens, q_lens, scale), o)
    return o, lse


CASES = [  # lens, q_lens, Nq, Hq, Hkv, D, page
    ([1], None, 1, 1, 1, 8, 1), ([0, 1, 2], None, 1, 2, 1, 64, 16), ([63, 64, 65, 0], None, 1, 8, 2, 128, 16),
    ([700], None, 1, 32, 8, 128, 24), ([5000, 3, 900], None, 1, 4, 4, 64, 64), ([40001], None, 1, 1, 1, 64, 128),
    ([130, 7, 4, 2], [5, 5, 4, 1], 5, 12, 4, 80, 24), ([17, 33, 3], [0, 4, 9], 4, 6, 2, 40, 7), ([300, 2], None, 8, 16, 2, 96, 8),
    ([90, 65], None, 16, 4, 2, 120, 3), ([200], None, 64, 2, 1, 56, 16), ([1000, 31], [64, 33], 64, 6, 2, 128, 16),
    ([11], None, 3, 48, 1, 72, 5), ([260], None, 1, 40, 1, 128, 16), ([9000, 100], [2, 2], 2, 3, 3, 128, 1),
    ([5] * 300, None, 1, 2, 1, 64, 4), ([(37 * i) % 400 for i in range(200)], None, 1, 4, 2, 32, 16)]


@pytest.mark.parametrize("case", CASES)
def test_lengths_heads_and_pages(case):
    lens, q_lens, Nq, Hq, Hkv, D, page = case
    kp, vp, table = cache(lens, page, Hkv, D)
    q = randn(len(lens), Nq, Hq, D, seed=2)
    both(q, kp, vp, table, dev(lens), None if q_lens is None else dev(q_lens))


def test_lengths_outside_their_range():
    """Negative lengths count as none, those behind the table as its all; so for the queries."""
    kp, vp, table = cache([40, 40, 40, 40], 8, 2, 64)
    q = randn(4, 3, 4, 64, seed=2)
    for k_lens, q_lens in (([-3, 1000, 40, 2], [-1, 9, 3, 3]), ([40, 39, 2, 1], [3, 3, 3, 3])):
        both(q, kp, vp, table, dev(k_lens), dev(q_lens))


@pytest.mark.parametrize("bad", [NAN, INF, -INF, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("D,Nq,page", [(64, 1, 16), (128, 5, 24), (80, 20, 7)])
def test_places_that_are_not_seen_hold_anything(bad, D, Nq, page):
    """Pages of nobody, rows behind a stream's length, and newer tokens than a query's own."""
    lens = [200, 65, Nq, 131]
    kp, vp, table = cache(lens, page, 2, D)
    q = randn(4, Nq, 4, D, seed=2)
    clean = reference(q, kp, vp, table, lens)
    live = torch.zeros(kp.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for t in range(n):
            live[int(table[b, t // page]), t % page] = True
    kp[~live], vp[~live] = bad, bad
    o, lse = hwp.paged_attention(q, kp, vp, table, dev(lens), with_lse=True)
    check(o, clean[0], clean[1], "o")
    check(lse, clean[2], clean[3], "lse")
    for b, n in enumerate(lens):  # the last token: only the last query sees it
        kp[int(table[b, (n - 1) // page]), (n - 1) % page] = bad
        vp[int(table[b, (n - 1) // page]), (n - 1) % page] = bad
    o, lse = hwp.paged_attention(q, kp, vp, table, dev(lens), with_lse=True)
    check(o[:, : Nq - 1], clean[0][:, : Nq - 1], clean[1][:, : Nq - 1], "o")
    check(lse[:, :, : Nq - 1], clean[2][:, :, : Nq - 1], clean[3][:, :, : Nq - 1], "lse")
    if bad == bad and abs(bad) < INF:
        return
    assert not bool(o[:, Nq - 1].isfinite().all())


@pytest.mark.parametrize("page", [1, 3, 6, 4])
@pytest.mark.parametrize("D", [64, 72])
def test_small_pages_in_any_layout(page, D):
    """Pools whose strides have rows in common, or only 8 elements, heads between tokens and broadcast heads: equal bits."""
    lens, H = [300, 129, 5], 3
    kp, vp, table = cache(lens, page, H, D)
    q = randn(3, 4, 6, D, seed=2)
    o, _ = both(q, kp, vp, table, dev(lens))
    P = kp.shape[0]
    for extra, order in ((8, (0, 1, 2, 3)), (0, (0, 2, 1, 3)), (D, (1, 0, 2, 3)), (24, (2, 0, 1, 3))):
        pools = []
        for x in (kp, vp):
            shape = [x.shape[i] for i in order]
            wide = torch.full((*shape[:2], shape[2] * D + extra), NAN, dtype=torch.bfloat16, device="cuda")
            y = wide[..., : shape[2] * D].unflatten(-1, (shape[2], D)).permute(*(order.index(i) for i in range(4)))
            assert y.shape == x.shape
            y.copy_(x)
            pools.append(y)
        assert torch.equal(hwp.paged_attention(q, *pools, table, dev(lens)), o)
    one = [x[:, :, :1].expand(P, page, H, D) for x in (kp, vp)]
    same = [x.contiguous() for x in one]
    assert torch.equal(hwp.paged_attention(q, *one, table, dev(lens)), hwp.paged_attention(q, *same, table, dev(lens)))
    # The last page and row of the pool, and pages that are not there.
    last = torch.full_like(table, P - 1)
    both(q, kp, vp, last, dev([page, 1, 0]))
    last[0, 0] = P
    o = hwp.paged_attention(q, kp, vp, last, dev([page, 1, 0]))
    assert bool(o[0, 3].isnan().all()) and bool(o[1, 3].isfinite().all())


@pytest.mark.parametrize("Nq,Hq", [(1, 2), (5, 8), (20, 8)])
@pytest.mark.parametrize("n", [40, 3000, 20000])
def test_infinite_values_that_all_see(Nq, Hq, n):
    """One gives its channel that infinity, two of different signs give NaN; other channels have what they have."""
    D, page = 64, 16
    kp, vp, table = cache([n], page, 2, D)
    q = randn(1, Nq, Hq, D, seed=2)
    want = reference(q, kp, vp, table, [n])
    for t, d, x in ((0, 3, INF), (7, 5, -INF), (1, 9, INF), (n - Nq, 9, -INF), (n // 2, 11, INF), (n // 2 - 1, 11, INF)):
        vp[int(table[0, t // page]), t % page, :, d] = x
    o = hwp.paged_attention(q, kp, vp, table, dev([n]))
    assert bool((o[..., 3] == INF).all()) and bool((o[..., 5] == -INF).all()) and bool((o[..., 11] == INF).all())
    assert bool(o[..., 9].isnan().all())
    rest = [d for d in range(D) if d not in (3, 5, 9, 11)]
    check(o[..., rest], want[0][..., rest], want[1][..., rest], "o")


def test_one_value_that_is_no_number_for_each_query():
    """Token t's value is NaN in channel t alone: query i has NaN in the channels of the tokens that it sees."""
    Nq, n, D = 16, 50, 64
    kp, vp, table = cache([n], 16, 1, D)
    q = randn(1, Nq, 4, D, seed=2)
    want = reference(q, kp, vp, table, [n])
    for t in range(n - Nq, n):
        vp[int(table[0, t // 16]), t % 16, 0, t] = NAN
    o = hwp.paged_attention(q, kp, vp, table, dev([n]))
    for i in range(Nq):
        seen = torch.zeros(D, dtype=torch.bool, device="cuda")
        seen[n - Nq: n - Nq + i + 1] = True
        assert bool(o[0, i][:, seen].isnan().all())
        err = (o[0, i].double() - want[0][0, i]).abs()[:, ~seen]
        assert bool((err <= want[1][0, i][:, ~seen]).all())


def test_keys_masked_through_a_channel():
    """Keys of -inf or the lowest number before and between keys whose scores lie at any level."""
    for low in (-INF, torch.finfo(torch.bfloat16).min):
        for level in (-150.0, 0.0, 90.0):
            for D, n, page in ((64, 400, 16), (128, 6000, 24)):
                kp, vp, table = cache([n], page, 2, D)
                q = randn(1, 1, 4, D, seed=2)
                kp *= 0.3
                q[..., 0], q[..., 1] = 1.0, 1.0
                kp[..., 0], kp[..., 1] = 0.0, level
                dead = [t for t in range(n) if t < n // 2 or t % 3 == 0]
                live = [t for t in range(n) if not (t < n // 2 or t % 3 == 0)]
                at = table[0, torch.tensor(live) // page].long(), torch.tensor(live, device="cuda") % page
                lk, lv = kp[at][None], vp[at][None]
                want = reference(q, lk, lv, dev([[0]]), [len(live)], scale=1.0)
                gone = table[0, torch.tensor(dead) // page].long(), torch.tensor(dead, device="cuda") % page
                kp[(*gone, slice(None), 0)] = low
                o, lse = hwp.paged_attention(q, kp, vp, table, dev([n]), scale=1.0, with_lse=True)
                check(o, want[0], want[1], "o")
                check(lse, want[2], want[3], "lse")
                kp[..., 0] = -INF
                o, lse = hwp.paged_attention(q, kp, vp, table, dev([n]), scale=1.0, with_lse=True)
                assert bool((o == 0).all()) and bool((lse == -INF).all())


@pytest.mark.parametrize("where", [0, 30, 62])
def test_numbers_that_are_none_in_seen_places_show(where):
    n, page = 1000, 16
    kp, vp, table = cache([n, 50], page, 2, 64)
    q = randn(2, 1, 4, 64, seed=2)
    fine = hwp.paged_attention(q, kp, vp, table, dev([n, 50]))
    kp[int(table[0, where]), 3, 1] = NAN
    o, lse = hwp.paged_attention(q, kp, vp, table, dev([n, 50]), with_lse=True)
    assert bool(o[0, :, 2:].isnan().all()) and bool(lse[0, 2:].isnan().all())
    assert torch.equal(o[0, :, :2], fine[0, :, :2]) and torch.equal(o[1], fine[1]) and bool(lse[1].isfinite().all())


@pytest.mark.parametrize("n", [100, 20000])
@pytest.mark.parametrize("entry", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_entries_outside_the_pool(n, entry):
    """A needed entry that is no page: that stream's queries are NaN (those with a token), the others are as they were."""
    lens = [300, n, 40]
    kp, vp, table = cache(lens, 16, 2, 64)
    q = randn(3, 3, 4, 64, seed=2)
    q_lens = dev([3, 2, 3])
    fine, fine_lse = hwp.paged_attention(q, kp, vp, table, dev(lens), q_lens, with_lse=True)
    table[1, n // 32] = entry
    table[2, 3:] = entry  # not needed
    o, lse = hwp.paged_attention(q, kp, vp, table, dev(lens), q_lens, with_lse=True)
    assert bool(o[1, :2].isnan().all()) and bool(lse[1, :, :2].isnan().all())
    assert bool((o[1, 2] == 0).all()) and bool((lse[1, :, 2] == -INF).all())
    for b in (0, 2):
        check(o[b], fine[b].double(), 2 * RB * fine[b].double().abs() + 1e-3, "o")
        assert bool((lse[b] - fine_lse[b]).abs().nan_to_num(0).max() < 1e-3)


def test_no_pages_at_all():
    kp = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = randn(2, 1, 4, 64)
    o, lse = hwp.paged_attention(q, kp, kp, dev([[], []]).view(2, 0), dev([0, 5]), with_lse=True)
    assert bool((o == 0).all()) and bool((lse == -INF).all())
    o = hwp.paged_attention(q, kp, kp, dev([[0], [0]]), dev([0, 5]))
    assert bool((o[0] == 0).all()) and bool(o[1].isnan().all())


@pytest.mark.parametrize("spread,scale", [(6.0, None), (1.0, 3.0), (1.0, -0.5), (1.0, 0.0)])
def test_large_scores_and_other_scales(spread, scale):
    lens = [900, 70]
    kp, vp, table = cache(lens, 16, 2, 128)
    both(randn(2, 2, 4, 128, seed=2, spread=spread), kp, vp, table, dev(lens), None, scale)


def test_layouts():
    """Heads before tokens in the pages, pools of their own, strided queries and outputs, wide table rows."""
    lens, page, Hq, Hkv, D = [130, 77], 16, 4, 2, 64
    kp, vp, table = cache(lens, page, Hkv, D)
    q = randn(2, 3, Hq, D, seed=2)
    o, lse = both(q, kp, vp, table, dev(lens))
    kt, vt = kp.transpose(1, 2).contiguous().transpose(1, 2), vp.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((2, table.shape[1] + 5), 10 ** 6, dtype=torch.int32, device="cuda")
    wide[:, 2: 2 + table.shape[1]] = table
    qkv = torch.full((2, 3, 3, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    qkv[:, :, 1] = q
    out = torch.full((2, Hq, 5, D), 7.0, dtype=torch.bfloat16, device="cuda")
    hwp.tok_paged_attention(qkv[:, :, 1], kt, vt, wide[:, 2: 2 + table.shape[1]], dev(lens), out.transpose(1, 2)[:, 1:4])
    assert torch.equal(out.transpose(1, 2)[:, 1:4], o)
    assert bool((out[:, :, 0] == 7).all()) and bool((out[:, :, 4] == 7).all())
    one = kp[:, :, :1].expand(-1, -1, Hkv, -1)  # one key head for all
    both(q, one, vp, table, dev(lens))
    both(q, kp, kp, table, dev(lens))           # values that are the keys
    same = table[:1].expand(2, -1).contiguous()  # two streams over the same pages
    both(q, kp, vp, same, dev([130, 130]))


def test_workspace_and_surroundings():
    lens, Hq, Hkv, D = [5000], 2, 1, 64
    kp, vp, table = cache(lens, 16, Hkv, D)
    q = randn(1, 2, Hq, D, seed=2)
    need = hwp.paged_attention_workspace_size(1, 2, Hq, Hkv, D)
    buf = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((1, 4, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    hwp.tok_paged_attention(q, kp, vp, table, dev(lens), out[:, 1:3], workspace=buf[256: 256 + need])
    assert torch.equal(out[:, 1:3], hwp.paged_attention(q, kp, vp, table, dev(lens)))
    assert bool((out[:, 0] == 3).all()) and bool((out[:, 3] == 3).all())
    assert bool((buf[:256] == 77).all()) and bool((buf[256 + need:] == 77).all())
    with pytest.raises(hwp.TokError) as e:
        hwp.tok_paged_attention(q, kp, vp, table, dev(lens), out[:, 1:3], workspace=buf[256: 256 + need - 16])
    assert e.value.status == hwp.TOK_ERR_SHAPE


def test_streams_graphs_and_empty_calls():
    sets = []
    for seed in (1, 2):
        lens = [3000 * seed, 50, 777]
        kp, vp, table = cache(lens, 16, 2, 128, seed=seed)
        sets.append((randn(3, 1, 8, 128, seed=seed + 5), kp, vp, table, dev(lens)))
    want = [hwp.paged_attention(*s, with_lse=True) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(hwp.paged_attention(*sets[i], with_lse=True, stream=s))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(w, r))
    q, kp, vp, table, lens = sets[0]
    sq, sl = torch.zeros_like(q), torch.zeros_like(lens)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            o, lse = hwp.paged_attention(sq, kp, vp, table, sl, with_lse=True)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((o == 0).all()) and bool((lse == -INF).all())
        sq.copy_(q), sl.copy_(lens)  # the lengths grow between replays
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert hwp.paged_attention(e(0, 1, 8, 128), kp, vp, table[:0], lens[:0]).numel() == 0
    assert hwp.paged_attention(e(3, 0, 8, 128), kp, vp, table, lens).numel() == 0
    del graph


def test_equals_cross_attention_without_pages():
    """One query over a batch's keys: the same call as cross attention's, up to both tolerances."""
    B, n, Hq, Hkv, D, page = 3, 512, 8, 2, 128, 64
    k, v, q = randn(B, n, Hkv, D), randn(B, n, Hkv, D, seed=2), randn(B, 1, Hq, D, seed=3)
    lens = dev([512, 100, 511])
    table = torch.arange(B * n // page, dtype=torch.int32, device="cuda").view(B, -1)
    want = reference(q, k.reshape(-1, page, Hkv, D), v.reshape(-1, page, Hkv, D), table, lens)
    for o in (hwp.cross_attention(q, k, v, lens),
              hwp.paged_attention(q, k.view(-1, page, Hkv, D), v.view(-1, page, Hkv, D), table, lens)):
        check(o, want[0], want[1], "o")


@pytest.mark.parametrize("n", [100, 20000])
@pytest.mark.parametrize("entry", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("Nq,Hq,page", [(3, 4, 16), (1, 2, 1), (20, 8, 24)])
def test_an_entry_outside_the_pool_reaches_no_other_stream(n, entry, Nq, Hq, page):
    """The other streams' outputs and lse are finite and have the bits that they have without it."""
    lens = [300, n, 40]
    kp, vp, table = cache(lens, page, 2, 64)
    q = randn(3, Nq, Hq, 64, seed=2)
    fine, fine_lse = hwp.paged_attention(q, kp, vp, table, dev(lens), with_lse=True)
    assert bool(fine.isfinite().all()) and bool(fine_lse.isfinite().all())
    table[1, n // 2 // page] = entry
    o, lse = hwp.paged_attention(q, kp, vp, table, dev(lens), with_lse=True)
    assert bool(o[1].isnan().all()) and bool(lse[1].isnan().all())
    for b in (0, 2):
        assert torch.equal(o[b], fine[b]) and torch.equal(lse[b], fine_lse[b])


@pytest.mark.parametrize("Nq,Hq", [(1, 2), (64, 4)])
@pytest.mark.parametrize("page,D", [(1, 64), (16, 64), (24, 128), (64, 128)])
def test_an_empty_pool(page, Nq, Hq, D):
    """No page: a query that would see a token is NaN, the others are 0, whatever the pool's strides and its null address."""
    kp = torch.empty(0, page, 2, D, dtype=torch.bfloat16, device="cuda")
    q = randn(3, Nq, Hq, D)
    lens = [0, 2 * page, 3]
    o, lse = hwp.paged_attention(q, kp, kp, dev([[0, -1, 5]] * 3), dev(lens), with_lse=True)
    for b, n in enumerate(lens):
        see = torch.arange(Nq, device="cuda") + n - Nq >= 0
        assert bool(o[b, see].isnan().all()) and bool(lse[b, :, see].isnan().all())
        assert bool((o[b, ~see] == 0).all()) and bool((lse[b, :, ~see] == -INF).all())


@pytest.mark.parametrize("Nq,Hq", [(1, 2), (5, 8), (20, 8)])
@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("n,at", [(40, 0), (40, 19), (3000, 2000), (20000, 0), (20000, 15000)])
def test_infinite_scores(Nq, Hq, D, n, at):
    """A key of infinity: queries with a positive channel there have NaN in both, those with a negative one do not count it."""
    page = 16
    kp, vp, table = cache([n], page, 1, D)
    q = randn(1, Nq, Hq, D, seed=2)
    q[..., 0] = q[..., 0].abs() + 1
    q[:, :, 1::2, 0] *= -1
    kp[int(table[0, at // page]), at % page, 0, 0] = INF
    o, lse = hwp.paged_attention(q, kp, vp, table, dev([n]), with_lse=True)
    assert bool(o[:, :, ::2].isnan().all()) and bool(lse[:, ::2].isnan().all())
    # The tokens but that one, as a cache of their own: the last queries' positions are the same.
    rest = torch.tensor([t for t in range(n) if t != at], device="cuda")
    where = table[0, rest // page].long(), rest % page
    want = reference(q, kp[where][None], vp[where][None], dev([[0]]), [n - 1])
    check(o[:, :, 1::2], want[0][:, :, 1::2], want[1][:, :, 1::2], "o")
    check(lse[:, 1::2], want[2][:, 1::2], want[3][:, 1::2], "lse")
