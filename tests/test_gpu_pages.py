"""Page tables, pages given back and writing into pages, against plain implementations on the host.  All exact."""
import random

import pytest
import torch

import haar_wavelet_patching_b200 as hwp

pytestmark = pytest.mark.gpu

I32 = torch.int32


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def plain_tables(lens, fresh, held, free, pages, table, N, M, page):
    """The rules, stream by stream: (slots, held, free, table, bad)."""
    held, table = list(held), [list(r) for r in table]
    free = min(max(free, 0), len(pages))
    slots, bad, asked, top = [], 0, 0, free
    for b, n in enumerate(lens):
        new = min(max(N if fresh is None else fresh[b], 0), N)
        held[b] = min(max(held[b], 0), M)
        row = [-1] * N
        if n < 0 or n + new > M * page:
            bad += 1
            slots.append(row)
            continue
        need = max(0, -(-(n + new) // page) - held[b])
        asked += need
        if need and asked > top:
            bad += 1
            slots.append(row)
            continue
        for _ in range(need):
            free -= 1
            table[b][held[b]] = pages[free]
            held[b] += 1
        for i in range(new):
            t = n + i
            s = table[b][t // page] * page + t % page
            row[i] = s if 0 <= s < 2 ** 31 and table[b][t // page] >= 0 else -1
        slots.append(row)
    return slots, held, free, table, bad


def plain_release(lens, held, free, pages, table, M, page):
    held, pages, table = list(held), list(pages), [list(r) for r in table]
    free = min(max(free, 0), len(pages))
    held = [min(max(h, 0), M) for h in held]
    keep = [min(h, -(-max(n, 0) // page)) for h, n in zip(held, lens)]
    back = sum(h - k for h, k in zip(held, keep))
    if back > len(pages) - free:
        return held, free, pages, table, 1
    at = free + back
    for b, (h, k) in enumerate(zip(held, keep)):
        for j in range(k, h):
            at -= 1
            pages[at] = table[b][j]
            table[b][j] = -1
    return keep, free + back, pages, table, 0


def state(rng, B, M, page, F, longest):
    """Streams that hold pages of a pool, the rest of them free, in any order."""
    pool = rng.sample(range(10 * F + 1), F)
    lens, held, table = [], [], []
    for b in range(B):
        h = min(M, rng.randint(0, longest) // page + rng.choice((0, 0, 1)))
        h = min(h, len(pool))
        lens.append(rng.randint(max(0, (h - 1) * page), h * page) if h else 0)
        held.append(h)
        table.append([pool.pop() for _ in range(h)] + [-7] * (M - h))
    return lens, held, table, pool + [-3] * (F - len(pool)), len(pool)


CASES = [  # B, N, M, page, F, longest
    (1, 1, 1, 1, 1, 0), (1, 5, 4, 16, 10, 30), (16, 5, 230, 16, 4000, 3000), (7, 0, 5, 8, 40, 20), (3, 100, 60, 2, 200, 30),
    (256, 40, 5, 24, 900, 50), (1025, 3, 3, 4, 2500, 6), (2100, 17, 9, 3, 4000, 9), (5, 900, 400, 7, 1500, 1000),
    (64, 8, 2, 128, 70, 100), (4, 3, 0, 16, 5, 0), (9, 2, 3, 1, 0, 0)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("seed", range(3))
def test_tables(case, seed):
    B, N, M, page, F, longest = case
    rng = random.Random(seed * 1000 + B)
    lens, held, table, pages, free = state(rng, B, M, page, F, longest)
    fresh = None if seed == 0 else [rng.randint(-1, N + 1) for _ in range(B)]
    if seed == 2 and B > 2:
        lens[1], lens[2] = -1, M * page + 1
    want = plain_tables(lens, fresh, held, free, pages, table, N, M, page)
    t, h, f, bad = dev(table).view(B, M), dev(held), dev([free]), dev([0])
    slots = torch.full((B, N), 9, dtype=I32, device="cuda")
    ho, fo = torch.full_like(h, 9), torch.full_like(f, 9)
    args = (dev(lens), None if fresh is None else dev(fresh), h, f, dev(pages), t)
    hwp.tok_page_tables(*args, slots, ho, fo, page, bad)
    assert (slots.tolist(), ho.tolist(), fo.item(), t.tolist(), bad.item()) == want
    assert h.tolist() == held and f.item() == free
    again = hwp.page_tables(args[0], args[1], N, h, f, args[4], t, page)  # in place; the same pages are taken
    assert torch.equal(again, slots) and torch.equal(h, ho) and torch.equal(f, fo) and t.tolist() == want[3]
    if want[4] == 0:  # nothing new the next time: the pages are there
        assert torch.equal(hwp.page_tables(args[0], args[1], N, h, f, args[4], t, page), slots) and f.item() == want[2]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("seed", range(2))
def test_release(case, seed):
    B, N, M, page, F, longest = case
    rng = random.Random(seed * 77 + B)
    lens, held, table, pages, free = state(rng, B, M, page, F, longest)
    less = [rng.choice((n, n // 2, 0, -1)) for n in lens]
    if seed == 1:
        pages = pages[: free + 1]  # room for one
    want = plain_release(less, held, free, pages, table, M, page)
    t, h, f, p, bad = dev(table).view(B, M), dev(held), dev([free]), dev(pages), dev([0])
    hwp.page_release(dev(less), h, f, p, t, page, bad)
    assert (h.tolist(), f.item(), p.tolist(), t.tolist(), bad.item()) == want


def test_taken_released_and_taken_again():
    """A round of drafts that is rolled back and taken again gives the same slots; so does one replayed from a graph."""
    rng = random.Random(3)
    B, N, M, page = 30, 6, 20, 4
    lens, held, table, pages, free = state(rng, B, M, page, 700, 50)
    t, h, f, p, n = dev(table), dev(held), dev([free]), dev(pages), dev(lens)
    first = hwp.page_tables(n, None, N, h, f, p, t, page)
    left = f.item()  # (what lies in the list behind the free pages is of no account)
    after = t.clone(), h.clone(), f.clone(), p[:left].clone()
    hwp.page_release(n, h, f, p, t, page)
    again = hwp.page_tables(n, None, N, h, f, p, t, page)
    assert torch.equal(first, again)
    assert all(torch.equal(a, b) for a, b in zip(after, (t, h, f, p[:left])))
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            hwp.page_release(n, h, f, p, t, page)
            third = hwp.page_tables(n, None, N, h, f, p, t, page)
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, third)
    assert all(torch.equal(a, b) for a, b in zip(after, (t, h, f, p[:left])))
    del graph


def test_counts_outside_their_range_and_odd_pages():
    """held and free beyond their arrays count as full; a page below 0 or a slot of 2^31 gives -1."""
    t = dev([[5, -2, 2 ** 30], [1, 2, 3]])
    slots = hwp.page_tables(dev([0, 0]), dev([9, 0]), 9, dev([77, -4]), dev([99]), dev([8, 9]), t, 3)
    assert slots.tolist() == [[15, 16, 17, -1, -1, -1, -1, -1, -1], [-1] * 9]
    free = dev([-5])
    slots = hwp.page_tables(dev([0]), None, 1, dev([0]), free, dev([8, 9]), dev([[0]]), 3)
    assert slots.tolist() == [[-1]] and free.item() == 0


def test_table_rows_inside_larger_ones():
    big = dev([[-1] * 9 for _ in range(4)])
    t = big[:, 2:5]
    slots = hwp.page_tables(dev([0] * 4), None, 5, dev([0] * 4), dev([8]), dev(range(8)), t, 4)
    assert t.tolist() == [[7 - 2 * b, 6 - 2 * b, -1] for b in range(4)]
    assert bool((big[:, :2] == -1).all()) and bool((big[:, 5:] == -1).all())
    assert slots[0].tolist() == [28, 29, 30, 31, 24]


def randn(*shape, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


WRITES = [(1, 1, 1, 8, 1, 1), (3, 5, 2, 64, 6, 16), (2, 700, 3, 128, 60, 24), (16, 5, 8, 128, 20, 16), (2, 33, 16, 80, 9, 8),
          (1, 300, 33, 96, 301, 1), (4, 0, 2, 64, 3, 4), (2, 3, 2, 64, 0, 4)]


@pytest.mark.parametrize("case", WRITES)
def test_write(case):
    B, N, H, D, P, page = case
    kv = randn(B, N, 2, H, D)  # slices of one projection
    pool = randn(P, 2, page, H, D, seed=2)
    want = pool.clone()
    rng = random.Random(B * N)
    order = rng.sample(range(P * page), min(P * page, B * N)) + [P * page + 3, 2 ** 31 - 1, -1, -2 ** 31] * (B * N)
    order = order[: B * N]
    rng.shuffle(order)
    slots, bad = dev(order).view(B, N), dev([0])
    hwp.paged_write(kv[:, :, 0], kv[:, :, 1], pool[:, 0], pool[:, 1], slots, bad)
    flat = kv.reshape(B * N, 2, H, D)
    for i, s in enumerate(order):
        if 0 <= s < P * page:
            want[s // page, :, s % page] = flat[i]
    assert torch.equal(pool, want)
    assert bad.item() == sum(s >= P * page for s in order)


def test_write_layouts():
    """Heads before tokens in the pages, one key head for all in the tokens, keys and values in pools of their own."""
    B, N, H, D, P, page = 2, 9, 4, 64, 5, 8
    k, v = randn(B, N, 1, D).expand(B, N, H, D), randn(B, H, N, D, seed=2).transpose(1, 2)
    kp, vp = (randn(P, H, page, D, seed=s).transpose(1, 2) for s in (3, 4))
    slots = dev(random.Random(1).sample(range(P * page), B * N)).view(B, N)
    wk, wv = kp.clone(), vp.clone()
    for b in range(B):
        for n in range(N):
            s = int(slots[b, n])
            wk[s // page, s % page], wv[s // page, s % page] = k[b, n], v[b, n]
    hwp.paged_write(k, v, kp, vp, slots)
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


def test_write_far_behind_2_31_elements():
    """The pool's last page lies more than 2^32 elements behind its first."""
    P, page, H, D = 17000, 128, 16, 128  # 2^32.05 elements, 8.9 GB
    pool = torch.empty(P, page, H, D, dtype=torch.bfloat16, device="cuda")
    pool[P - 1].zero_()
    kv = randn(1, 2, H, D)
    v_pool = torch.empty_like(pool)
    v_pool[P - 1].zero_()
    slots = dev([[P * page - 1, P * page - 7]])
    hwp.paged_write(kv, 2 * kv, pool, v_pool, slots)
    assert torch.equal(pool[P - 1, page - 1], kv[0, 0]) and torch.equal(pool[P - 1, page - 7], kv[0, 1])
    assert torch.equal(v_pool[P - 1, page - 1], 2 * kv[0, 0])
    table = dev([[P - 1]])
    q = randn(1, 1, H, D, seed=5)
    o = hwp.paged_attention(q, pool, v_pool, table, dev([page]))
    near = hwp.paged_attention(q, pool[P - 1:].clone(), v_pool[P - 1:].clone(), dev([[0]]), dev([page]))
    assert torch.equal(o, near)


@pytest.mark.parametrize("free,F", [(7, 9), (12, 9), (-3, 9), (0, 0)])
def test_without_streams_the_count_is_still_written(free, F):
    """B = 0: nothing is taken or given back, and free_out gets the count, in place or into another tensor."""
    none, table, pages = dev([]), torch.empty(0, 5, dtype=I32, device="cuda"), dev(range(F))
    want = min(max(free, 0), F)
    for in_place in (False, True):
        f = dev([free])
        fo = f if in_place else dev([99])
        slots = torch.empty(0, 3, dtype=I32, device="cuda")
        hwp.tok_page_tables(none, None, none, f, pages, table, slots, none, fo, 4)
        assert fo.item() == want
        f = dev([free])
        fo = f if in_place else dev([99])
        hwp.tok_page_release(none, none, f, pages, table, none, fo, 4)
        assert fo.item() == want and (in_place or f.item() == free)
        assert pages.tolist() == list(range(F))
