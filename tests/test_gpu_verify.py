"""Verifying drafted codes against a 64-bit implementation on the host: codes and counts are equal."""
import numpy as np
import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def probabilities(x, t):
    """Weights over the codes, adding up to 1 (or all 0)."""
    x = np.where(np.isnan(x), -INF, x)
    w = np.zeros(x.shape)
    if x.max() == -INF:
        return w
    if not t > 0:
        w[int(np.argmax(x))] = 1.0
    elif x.max() == INF:
        w[x == INF] = 1.0
    else:
        with np.errstate(under="ignore"):
            w = np.exp((x - x.max()) / min(t, 3.4e38))
    return w / w.sum()


def plain(logits, codes, u, draft=None, n_draft=None, temperature=1.0):
    logits = logits.double().cpu().numpy()
    draft = None if draft is None else draft.double().cpu().numpy()
    codes, u = codes.cpu().numpy(), u.double().cpu().numpy()
    B, K, V = logits.shape[0], logits.shape[1] - 1, logits.shape[2]
    t = np.broadcast_to(np.asarray(temperature.double().cpu() if torch.is_tensor(temperature) else np.float32(temperature), dtype=np.float64), (B,))
    u = np.clip(np.where(np.isnan(u), 0.0, u), 0.0, 1 - 2.0 ** -24)
    out, accepted = np.full((B, K + 1), -1, dtype=np.int64), np.zeros(B, dtype=np.int64)
    for b in range(B):
        n = K if n_draft is None else min(max(int(n_draft[b]), 0), K)
        i = 0
        while True:
            p = probabilities(logits[b, i], t[b])
            r = p
            if i < n:
                x = int(codes[b, i])
                inside = 0 <= x < V
                q = np.zeros(V)
                if draft is not None:
                    q = probabilities(draft[b, i], t[b])
                elif inside:
                    q[x] = 1.0
                if inside and u[b, i] * q[x] < p[x]:
                    out[b, i] = x
                    i += 1
                    continue
                r = np.maximum(p - q, 0.0)
                r = r if r.sum() > 0 else p
            c = np.cumsum(r)
            if c[-1] > 0:
                at = min(int(np.searchsorted(c, u[b, K] * c[-1], side="right")), V - 1)
                while r[at] == 0:  # (rounding: the last one with a weight)
                    at -= 1
                out[b, i] = at
            accepted[b] = i
            break
    return out, accepted


def data(B, K, V, dtype=F32, spread=2.0, noise=0.5, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(B, K + 1, V, generator=g, device="cuda") * spread
    draft = (logits[:, :K] + torch.randn(B, K, V, generator=g, device="cuda") * noise).to(dtype)
    gumbel = -(-torch.rand(B, K, V, generator=g, device="cuda").clamp_min(1e-30).log()).log()
    codes = (draft.float() + gumbel).argmax(2).to(torch.int32) if K else torch.zeros(B, 0, dtype=torch.int32, device="cuda")
    return logits.to(dtype), draft, codes, torch.rand(B, K + 1, generator=g, device="cuda")


def check(logits, codes, u, draft=None, n_draft=None, temperature=1.0):
    out, accepted = hwp.verify_codes(logits, codes, u, draft, n_draft, temperature)
    want, count = plain(logits, codes, u, draft, n_draft, temperature)
    assert accepted.tolist() == count.tolist()
    assert out.tolist() == want.tolist()
    return out, accepted


@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (1, 1, 1), (3, 2, 2), (2, 4, 7), (5, 3, 1000), (1, 63, 300), (4, 4, 64000), (16, 5, 8001),
                                   (40, 2, 4097), (90, 3, 64000), (300, 2, 513), (700, 1, 2000), (1, 4, 262144)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("point", [False, True])
def test_sizes(B, K, V, dtype, point):
    logits, draft, codes, u = data(B, K, V, dtype)
    check(logits, codes, u, None if point else draft, None, 0.9)


@pytest.mark.parametrize("spread,noise,temperature", [(0.1, 0.05, 1.0), (4.0, 3.0, 0.5), (2.0, 0.01, 1.3), (3.0, 1.0, 0.0), (3.0, 1.0, -1.0),
                                                      (2.0, 0.5, 1e-8), (2.0, 0.5, 1e30), (2.0, 0.5, INF), (2.0, 0.5, float("nan"))])
@pytest.mark.parametrize("B", [3, 200])
def test_spreads_and_temperatures(spread, noise, temperature, B):
    for dtype in (F32, BF16):
        logits, draft, codes, u = data(B, 4, 3001, dtype, spread, noise)
        check(logits, codes, u, draft, None, temperature)
        check(logits, codes, u, None, None, temperature)


@pytest.mark.parametrize("offset", [0.0, 700.0, -1900.0, 2100.0, -1e5, 1e12])
@pytest.mark.parametrize("temperature", [0.01, 0.9, 40.0])
def test_rows_far_from_zero(offset, temperature):
    """The weights are the differences' alone, on both sides of where these are taken before the product with 1 / T."""
    logits, draft, codes, u = data(6, 3, 4001, F32, 5.0 * temperature, 1.0)
    logits[1::2] += offset
    draft[::2] -= offset
    check(logits, codes, u, draft, None, temperature)
    check(logits, codes, u, None, None, temperature)


def test_counts_and_temperatures_per_stream():
    B, K, V = 12, 5, 2000
    logits, draft, codes, u = data(B, K, V)
    n = torch.tensor([(i % 9) - 1 for i in range(B)], dtype=torch.int32, device="cuda")
    t = torch.linspace(0.0, 2.0, B, device="cuda")
    check(logits, codes, u, draft, n, t)
    check(logits, codes, u, None, n, t)


def test_drafts_of_the_model_itself_all_stand():
    """p = q: u q < p for every u in (0, 1); the code behind is drawn from the last row."""
    logits, _, codes, u = data(8, 6, 5000)
    u.clamp_(1e-6, 1 - 1e-6)
    out, accepted = check(logits, codes, u, logits[:, :6])
    assert bool((accepted == 6).all()) and torch.equal(out[:, :6], codes)


def test_nothing_left_and_numbers_at_the_ends():
    V = 50
    for value in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan")):
        logits, draft, codes, u = data(6, 3, V)
        u[:] = value
        check(logits, codes, u, draft)
        check(logits, codes, u)
    # one certain code, and another one drafted for certain; the same one drafted and refused by no number
    logits = torch.full((2, 2, V), -INF, device="cuda")
    logits[:, :, 7] = 3.0
    codes = torch.tensor([[7], [9]], dtype=torch.int32, device="cuda")
    u = torch.full((2, 2), 0.5, device="cuda")
    out, accepted = check(logits, codes, u)
    assert out.tolist() == [[7, 7], [7, -1]] and accepted.tolist() == [1, 0]


def test_special_logits_and_codes():
    V = 300
    logits, draft, codes, u = data(16, 3, V, seed=4)
    nan = float("nan")
    logits[0, 1] = -INF                      # nothing to draw from
    logits[1, 0, 5:9] = INF                  # only these count
    logits[2, :, ::2] = nan
    draft[3, 0] = -INF                       # the draft gives nothing a probability
    draft[4, 1, 17] = INF
    codes[4, 1] = 17
    draft[5, :, 100:] = nan
    codes[6, 0], codes[7, 1], codes[8, 2], codes[9, 0] = -1, V, 2 ** 31 - 1, -2 ** 31
    logits[10, 0], draft[10, 0] = -INF, -INF
    logits[11, 0, 3], draft[11, 0, 3] = INF, INF
    codes[11, 0] = 3
    logits[12], draft[12] = torch.finfo(F32).min, torch.finfo(F32).min
    logits[13] = torch.finfo(F32).max
    logits[14, :, 1], logits[14, :, 2] = torch.finfo(F32).max, torch.finfo(F32).min
    for t in (1.0, 0.0, 0.3):
        check(logits, codes, u, draft, None, t)
        check(logits, codes, u, None, None, t)


def test_tests_next_to_their_border():
    """u on either side of p / q by a little more than 64 bits tell apart, where 32 bits leave doubt."""
    logits, draft, codes, u = data(64, 1, 4000, noise=1.0)
    p, q = (torch.softmax(x[:, 0].double(), 1).gather(1, codes.long())[:, 0] for x in (logits, draft))
    ratio = (p / q).float()
    fits = (ratio < 1) & (ratio > 0)
    for step in (-1, 1):
        v = torch.nextafter(ratio, ratio + step)
        u[:, 0] = torch.where(fits, v, u[:, 0])
        far = ((v.double() * q - p).abs() > 1e-12 * p) | ~fits
        assert bool(far.any())
        check(logits[far], codes[far], u[far], draft[far])


def test_strides_and_addresses():
    B, K, V = 3, 2, 1001
    for dtype in (F32, BF16):
        logits, draft, codes, u = data(B, K, V, dtype)
        want = check(logits, codes, u, draft)
        big = torch.zeros(K + 1, B, V + 7, dtype=dtype, device="cuda")
        for shift in (0, 1, 3):
            x = big[:, :, shift: shift + V].transpose(0, 1)
            x.copy_(logits)
            both = torch.zeros(B, 2, K, V + 1, dtype=dtype, device="cuda")
            both[:, 1, :, 1:] = draft
            got = hwp.verify_codes(x, codes, u, both[:, 1, :, 1:])
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        one = logits[:1].expand(B, K + 1, V)
        check(one, codes, u, draft[:, :1].expand(B, K, V))


def test_distribution():
    """Drafts and their verification together draw from the model's distribution."""
    V, n = 5, 40000
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(1, 2, V, generator=g, device="cuda").expand(n, 2, V)
    draft = torch.randn(1, 1, V, generator=g, device="cuda").expand(n, 1, V)
    q = torch.softmax(draft[0, 0].double(), 0)
    p = torch.softmax(logits[0, 0].double(), 0)
    codes = torch.multinomial(q, n, replacement=True, generator=g).to(torch.int32)[:, None]
    u = torch.rand(n, 2, generator=g, device="cuda")
    out, _ = hwp.verify_codes(logits, codes, u, draft)
    freq = torch.bincount(out[:, 0].long(), minlength=V).double() / n
    assert bool(((freq - p).abs() < 5 * (p * (1 - p) / n).sqrt()).all())  # five standard deviations


def test_graph_streams_repeat_and_empty():
    logits, draft, codes, u = data(6, 4, 9000, BF16)
    want = hwp.verify_codes(logits, codes, u, draft)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [hwp.verify_codes(logits, codes, u, draft, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(want, r))
    su = torch.zeros_like(u)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            r = hwp.verify_codes(logits, codes, su, draft)
        su.copy_(u)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, r))
    out, accepted = hwp.verify_codes(logits[:0], codes[:0], u[:0], draft[:0])
    assert out.shape == (0, 5) and accepted.shape == (0,)
    del graph


@pytest.mark.parametrize("B,K,V", [(1, 1, 9), (5, 63, 40), (7, 3, 40000)])
def test_workspace_and_surroundings(B, K, V):
    """A workspace of just the size that is asked for, whatever lies in it; nothing beside it and the outputs is written."""
    logits, draft, codes, u = data(B, K, V)
    want = hwp.verify_codes(logits, codes, u, draft)
    need = hwp.verify_codes_workspace_size(B, K, V)
    for fill in (0, 255):
        ws = torch.full((need + 32,), fill, dtype=torch.uint8, device="cuda")
        out = torch.full((B + 2, K + 1), -7, dtype=torch.int32, device="cuda")
        accepted = torch.full((B + 2,), -7, dtype=torch.int32, device="cuda")
        hwp.tok_verify_codes(logits, codes, u, out[1:-1], accepted[1:-1], draft, workspace=ws[16: 16 + need])
        assert torch.equal(out[1:-1], want[0]) and torch.equal(accepted[1:-1], want[1])
        assert bool((ws[:16] == fill).all()) and bool((ws[16 + need:] == fill).all())
        assert all(bool((x[i] == -7).all()) for x in (out, accepted) for i in (0, -1))
    with pytest.raises(hwp.TokError):
        hwp.tok_verify_codes(logits, codes, u, *want, draft, workspace=ws[16: 16 + need - 1])


def test_follows_sample_codes_without_drafts():
    """K = 0 is a plain draw: sample_codes' without filters."""
    logits, _, codes, u = data(20, 0, 64000)
    out, accepted = hwp.verify_codes(logits, codes, u, temperature=0.8)
    assert torch.equal(out[:, 0], hwp.sample_codes(logits[:, 0], u[:, 0], temperature=0.8)) and not bool(accepted.any())
