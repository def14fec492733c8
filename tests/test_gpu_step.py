"""The operators of a step as a decoder uses them: codes in, their rows, rotary positions, room in the pages, keys and
values into it, attention over the pages, logits, verification, and the pages of refused drafts back.

Each step's attention is held against a 64-bit one over keys and values that the test keeps per stream (within the bound
of the attention's own tests), its codes against 64-bit verification of the same logits (equal), the pages against counting.
"""
import random

import pytest
import torch

import haar_wavelet_patching_b200 as hwp
from test_gpu_paged_attention import check, reference
from test_gpu_verify import plain

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
V, WIDTH, HQ, HKV, D = 211, 48, 6, 2, 40
LONGEST, K = 256, 3


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Decoder:
    """One layer; products in a fixed order, so that a captured step gives the bits of an eager one."""

    def __init__(self, B, page, spare, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
        self.rows = w(V, WIDTH)
        self.wq, self.wk, self.wv = w(WIDTH, HQ * D) * 0.3, w(WIDTH, HKV * D) * 0.3, w(WIDTH, HKV * D) * 0.2
        self.wo, self.guess = w(HQ * D, V) * 0.2, w(V, V)
        self.rope = hwp.rope_table((LONGEST, 1, 1), (D, 0, 0))
        self.page, M = page, -(-LONGEST // page)
        F = B * M // 2 + spare
        pool = torch.full((F, 2, page, HKV, D), float("nan"), dtype=BF16, device="cuda")
        self.kp, self.vp = pool[:, 0], pool[:, 1]
        self.pages = dev(random.Random(seed).sample(range(F), F))
        self.free, self.held, self.lens = dev([F]), dev([0] * B), dev([0] * B)
        self.table = dev([[-1] * M] * B)
        self.bad = dev([0])

    def state(self):
        return self.pages, self.free, self.held, self.lens, self.table, self.kp, self.vp, self.bad

    def step(self, new, fresh):
        """new [B, N] codes of which fresh [B] count: (q, k, v, o, logits [B, N, V])."""
        B, N = new.shape
        x = hwp.embed_codes(new, self.rows, 0.5, self.bad).float()
        q, k, v = ((x[..., None] * m.float()).sum(-2).to(BF16).view(B, N, -1, D) for m in (self.wq, self.wk, self.wv))
        pos = torch.zeros(B, N, 3, dtype=I32, device="cuda")
        pos[..., 0] = (self.lens[:, None] + torch.arange(N, device="cuda", dtype=I32)).clamp(max=LONGEST - 1)
        q, k = (hwp.rope_positions(t, pos, self.rope, (LONGEST, 1, 1), (D, 0, 0)) for t in (q, k))
        slots = hwp.page_tables(self.lens, fresh, N, self.held, self.free, self.pages, self.table, self.page, self.bad)
        hwp.paged_write(k, v, self.kp, self.vp, slots, self.bad)
        o = hwp.paged_attention(q, self.kp, self.vp, self.table, self.lens + fresh, fresh)
        logits = (o.reshape(B, N, HQ * D, 1).float() * self.wo.float()).sum(-2).to(BF16)
        return q, k, v, o, logits

    def keep(self, lens):
        """Tokens from lens [B] on are dropped and their pages given back."""
        self.lens.copy_(lens)
        hwp.page_release(self.lens, self.held, self.free, self.pages, self.table, self.page, self.bad)

    def drafts(self, last, u, temperature):
        """K codes drawn behind `last` [B] with u [B, K], and the logits that they are from."""
        codes, logits = [], []
        for i in range(K):
            logits.append(self.guess[last.long()])
            last = hwp.sample_codes(logits[-1], u[:, i].contiguous(), temperature)
            codes.append(last)
        return torch.stack(codes, 1).contiguous(), torch.stack(logits, 1).contiguous()

    def round(self, last, u, n_draft, active, temperature):
        """Drafts behind `last`, their verification, and what is refused taken back: (step's tensors, out, accepted, ...)."""
        codes, guesses = self.drafts(last, u[:, :K], temperature)
        got = self.step(torch.cat([last[:, None], codes], 1).contiguous(), (n_draft + 1) * active)
        # What the draft's model would want of the next code, too: so that some drafts stand.
        logits = (got[4].float() * 0.3 + self.guess[torch.cat([last[:, None], codes], 1).long()].float()).to(BF16)
        out, accepted = hwp.verify_codes(logits, codes, u[:, K:].contiguous(), guesses, n_draft, temperature)
        kept = self.lens + (accepted + 1) * active
        before = self.lens.clone()
        self.keep(kept)
        return got, logits, codes, guesses, out, accepted, before


def consistent(d, lens):
    """Every stream has the pages of its tokens and no more; no page twice, none lost."""
    held, table, free = d.held.tolist(), d.table.tolist(), d.free.item()
    assert held == [-(-n // d.page) for n in lens]
    own = [p for row, h in zip(table, held) for p in row[:h]]
    assert all(p == -1 for row, h in zip(table, held) for p in row[h:])
    assert sorted(own + d.pages[:free].tolist()) == list(range(d.kp.shape[0]))
    assert d.bad.item() == 0


@pytest.mark.parametrize("page,seed", [(1, 1), (4, 2), (16, 3), (24, 4)])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_prompts_then_rounds_of_drafts(page, seed, temperature):
    prompts = [5, 70, 1, 33]
    B, rng = len(prompts), random.Random(seed)
    d = Decoder(B, page, 8, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kept = [[torch.zeros(0, HKV, D, dtype=BF16, device="cuda")] * 2 for _ in range(B)]

    def looked_over(got, fresh, lens):
        q, k, v, o, _ = got
        for b in range(B):
            kept[b] = [torch.cat([t[: lens[b]], x[b, : fresh[b]]]) for t, x in zip(kept[b], (k, v))]
        most = max(t[0].shape[0] for t in kept)
        flat = torch.zeros(2, B, most, HKV, D, dtype=BF16, device="cuda")
        for b in range(B):
            for i in range(2):
                flat[i, b, : kept[b][i].shape[0]] = kept[b][i]
        want = reference(q, flat[0], flat[1], dev([[b] for b in range(B)]), dev([n + f for n, f in zip(lens, fresh)]), dev(fresh))
        for b in range(B):
            check(o[b, : fresh[b]], want[0][b, : fresh[b]], want[1][b, : fresh[b]], f"o of stream {b}")

    # Prompts, 32 tokens at a time.
    codes = dev([[rng.randrange(V) for _ in range(96)] for _ in range(B)])
    last = codes[torch.arange(B), torch.tensor(prompts) - 1].clone()
    lens = [0] * B
    for c in range(0, 96, 32):
        fresh = [max(0, min(32, n - 1 - c)) for n in prompts]
        got = d.step(codes[:, c: c + 32].contiguous(), dev(fresh))
        looked_over(got, fresh, lens)
        lens = [n + f for n, f in zip(lens, fresh)]
        d.keep(dev(lens))
        consistent(d, lens)
    # Rounds: ragged drafts, a stream that has ended from the third on.
    stood = 0
    for r in range(6):
        n_draft = [rng.randrange(K + 1) for _ in range(B)]
        active = [1] * B if r < 2 else [1, 1, 0, 1]
        u = torch.rand(B, 2 * K + 1, generator=g, device="cuda")
        got, logits, codes, guesses, out, accepted, before = d.round(last, u, dev(n_draft), dev(active), temperature)
        assert before.tolist() == lens
        looked_over(got, [(n + 1) * a for n, a in zip(n_draft, active)], lens)
        want, count = plain(logits, codes, u[:, K:], guesses, n_draft, temperature)
        assert accepted.tolist() == count.tolist() and out.tolist() == want.tolist()
        stood += sum(count)
        lens = [n + (int(c) + 1) * a for n, c, a in zip(lens, count, active)]
        assert d.lens.tolist() == lens
        consistent(d, lens)
        last = out.gather(1, accepted.long()[:, None])[:, 0].contiguous()
    assert stood > 0
    d.keep(dev([0] * B))
    consistent(d, [0] * B)


def test_a_captured_round_is_an_eager_one():
    """The same rounds, eager and replayed from a graph: equal bits, caches and tables included."""
    B, page, T = 3, 4, 0.9
    eager, graphed = Decoder(B, page, 0, 7), Decoder(B, page, 0, 7)
    g = torch.Generator(device="cuda").manual_seed(7)
    us = [torch.rand(B, 2 * K + 1, generator=g, device="cuda") for _ in range(5)]
    n_draft, active, last = dev([3, 0, 2]), dev([1, 1, 1]), dev([5, 6, 7])
    u, into = us[0].clone(), last.clone()

    def turn(d, last, u):
        r = d.round(last, u, n_draft, active, T)
        return r[3], r[4], r[5], r[0][3], r[4].gather(1, r[5].long()[:, None])[:, 0].contiguous()

    start = [t.clone() for t in graphed.state()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        turn(graphed, into, u)  # (warm)
        for t, s in zip(graphed.state(), start):
            t.copy_(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            result = turn(graphed, into, u)
            into.copy_(result[4])
        into.copy_(last)
    torch.cuda.synchronize()
    for r in range(5):
        u.copy_(us[r])
        graph.replay()
        want = turn(eager, last, us[r])
        last = want[4]
        torch.cuda.synchronize()
        for a, b in zip(want, result):
            assert torch.equal(a, b)
        live = int(eager.free.item())
        for name, a, b in zip(("pages", "free", "held", "lens", "table", "k", "v", "bad"), eager.state(), graphed.state()):
            if name == "pages":
                a, b = a[:live], b[:live]
            assert torch.equal(torch.nan_to_num(a.float(), nan=-7.0), torch.nan_to_num(b.float(), nan=-7.0)), name
    del graph
