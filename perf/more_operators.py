"""Cases of the operators of a token-by-token step over the codes: embedding of codes and its gradient, page tables
of the streams, writing keys and values into pages, attention of new tokens over the pages, and verification of
drafted codes.

`run` computes a case either in its plain form (elementary torch operations) or, with
`own` true, through this package's entry points; both take what `prepare` made.
"""
import math

import numpy as np
import torch

own = False

CODES = 64000  # FSQ codebook, levels (8, 8, 8, 5, 5, 5)


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def listed():
    return [
        # Next-token step of 16 streams, four drafted codes and the last one each.
        {"name": "embed_step", "op": "embed", "tokens": 80, "v": CODES, "d": 2048, "dtype": "bf16", "train": False,
         "hot": 0.0, "scale": 1.0},
        # Training step on the 121-frame 704x1280 clip's 16x44x80 latent grid: all tokens, the table's gradient.
        {"name": "embed_train_clip", "op": "embed", "tokens": 56320, "v": CODES, "d": 2048, "dtype": "bf16", "train": True,
         "hot": 0.0, "scale": 45.25},
        # A small odd grid (7x33x45) in fp32, a width that is no power of two, a tenth of the tokens the same code.
        {"name": "embed_train_odd", "op": "embed", "tokens": 10395, "v": CODES, "d": 1004, "dtype": "f32", "train": True,
         "hot": 0.1, "scale": 1.0},
        # Step of 16 streams with five new tokens each: few of them need another page.
        {"name": "tables_step", "op": "tables", "b": 16, "n": 5, "longest": 3520, "page": 16, "short": False},
        # Prompts of 256 streams join at once: up to a quarter of a frame each, odd pages.
        {"name": "tables_prompts", "op": "tables", "b": 256, "n": 880, "longest": 0, "page": 24, "short": False},
        # Keys and values of a step's tokens into the pages.
        {"name": "write_step", "op": "write", "b": 16, "n": 5, "longest": 3520, "page": 16, "heads": 8, "d": 128},
        # Keys and values of a frame (44x80) for 8 streams, into pages that other streams' lie between.
        {"name": "write_frame", "op": "write", "b": 8, "n": 3520, "longest": 3520, "page": 64, "heads": 8, "d": 128},
        # Next-token step of 16 streams, up to a frame in the cache (ragged), four query heads to a key head.
        {"name": "paged_step", "op": "paged", "b": 16, "n": 1, "longest": 3520, "page": 16, "hq": 32, "hkv": 8, "d": 128,
         "ragged": True, "empty": False},
        # Drafted step: up to five new tokens a stream, a head size between the tiles' sizes, odd pages, a stream that has ended.
        {"name": "paged_drafts_odd", "op": "paged", "b": 6, "n": 5, "longest": 7001, "page": 24, "hq": 12, "hkv": 4, "d": 80,
         "ragged": True, "empty": True},
        # Next-token step late in four clips: 16x44x80 tokens in the cache each.
        {"name": "paged_clip", "op": "paged", "b": 4, "n": 1, "longest": 56320, "page": 64, "hq": 32, "hkv": 8, "d": 128,
         "ragged": False, "empty": False},
        # Four drafted codes each of 4 streams.
        {"name": "verify_step", "op": "verify", "b": 4, "k": 4, "v": CODES, "dtype": "bf16", "point": False, "ragged": False,
         "temperature": 0.8, "spread": 2.5, "noise": 0.7},
        # A batch of streams with six drafted codes at most, fp32 logits.
        {"name": "verify_batch", "op": "verify", "b": 96, "k": 6, "v": CODES, "dtype": "f32", "point": False, "ragged": True,
         "temperature": 1.0, "spread": 2.0, "noise": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("embed", "embed", "grad", "grad", "tables", "write", "paged", "paged", "paged", "verify", "verify"))
    if kind in ("embed", "grad"):
        while True:
            c = {"op": "embed", "tokens": _log(rng, 1, 100000), "v": rng.choice((CODES, CODES, rng.randint(100, 65000))),
                 "d": rng.choice((64, 512, 1024, 2048, 4096, rng.randint(16, 600), 4 * rng.randint(20, 600))),
                 "dtype": rng.choice(("bf16", "bf16", "f32")), "train": kind == "grad",
                 "hot": rng.choice((0.0, 0.0, 0.05, 0.9)), "scale": rng.choice((1.0, 1.0, 22.6))}
            if work(c)["bytes"] <= 900e6 and c["v"] * c["d"] <= CODES * 2048:
                return c
    if kind == "tables":
        return {"op": "tables", "b": _log(rng, 1, 512), "n": _log(rng, 1, 880), "longest": rng.choice((0, 300, 3520)),
                "page": rng.choice((1, 8, 16, 24, 64, 128)), "short": rng.random() < 0.3}
    if kind == "write":
        while True:
            c = {"op": "write", "b": _log(rng, 1, 64), "n": _log(rng, 1, 3520), "longest": rng.choice((0, 300, 3520)),
                 "page": rng.choice((1, 16, 24, 64)), "heads": rng.randint(1, 16), "d": rng.choice((32, 64, 80, 96, 128))}
            if work(c)["bytes"] <= 230e6:
                return c
    if kind == "paged":
        while True:
            hkv, g = rng.randint(1, 16), rng.choice((1, 1, 2, 3, 4, 8, 16))
            c = {"op": "paged", "b": _log(rng, 1, 64), "n": rng.choice((1, 1, 1, 2, 4, 5, 8, 16)), "longest": _log(rng, 20, 60000),
                 "page": rng.choice((1, 8, 16, 24, 64, 128)), "hq": hkv * g, "hkv": hkv,
                 "d": rng.choice((32, 64, 64, 80, 96, 128, 128)), "ragged": rng.random() < 0.6, "empty": rng.random() < 0.3}
            c["empty"] = c["empty"] and c["b"] > 1
            if c["longest"] * c["b"] * hkv * c["d"] <= 4 * 56320 * 8 * 128 and work(c)["flops"] <= 16e9:
                return c
    return {"op": "verify", "b": _log(rng, 1, 48), "k": rng.choice((0, 1, 2, 4, 5, 8)),
            "v": rng.choice((CODES, CODES, rng.randint(300, 2000), rng.randint(2000, 65000))),
            "dtype": rng.choice(("bf16", "f32")), "point": rng.random() < 0.4, "ragged": rng.random() < 0.4,
            "temperature": rng.choice((0.0, 0.7, 1.0, 1.3)), "spread": rng.choice((0.5, 2.0, 4.0)),
            "noise": rng.choice((0.1, 0.5, 2.0))}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lens(case):
    """Tokens in each stream's cache: full, then shorter and shorter; the last one none where the case says so."""
    b, n = case["b"], case["longest"]
    lens = [-(-n * (b - i) // b) if case["ragged"] else n for i in range(b)]
    if case["empty"]:
        lens[-1] = 0
    return lens


def _news(case, lens):
    """New tokens of each stream among `lens`: all, or one to all."""
    n = case["n"]
    return [min(x, 1 + (5 * i + n - 1) % n if case["ragged"] else n) for i, x in enumerate(lens)]


def _drafts(case):
    return [(i * 5 + case["k"]) % (case["k"] + 1) if case["ragged"] else case["k"] for i in range(case["b"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev).to(dtype)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    def shuffled(n):
        return torch.randperm(n, generator=gen, device=dev).to(torch.int32)

    s = {"case": case}
    op = case["op"]
    if op == "embed":
        n, v, d = case["tokens"], case["v"], case["d"]
        used = torch.rand(n, generator=gen, device=dev, dtype=torch.float64)
        codes = (v * used * used).to(torch.int32).clamp_max(v - 1)  # codes are not equally frequent
        codes = torch.where(torch.rand(n, generator=gen, device=dev) < case["hot"], v // 2, codes).to(torch.int32)
        s["codes"], s["table"] = codes, normal(v, d, dtype=_type(case))
        if case["train"]:
            s["go"] = normal(n, d, dtype=_type(case))
        return s
    if op in ("tables", "write"):
        b, n, page = case["b"], case["n"], case["page"]
        s["lens"] = whole(0, case["longest"] + 1, b)
        s["new"] = whole(max(1, n // 2), n + 1, b)
        s["held"] = (s["lens"] + (page - 1)) // page
        width = (case["longest"] + n + page - 1) // page
        need = (s["lens"] + s["new"] + page - 1) // page - s["held"]
        total = b * width
        order = shuffled(total)
        column = torch.arange(width, device=dev)
        s["table"] = torch.where(column < s["held"][:, None], order.view(b, width), -1).to(torch.int32)
        spare = order.view(b, width)[column >= s["held"][:, None]]
        s["pages"] = torch.zeros(total, dtype=torch.int32, device=dev)
        s["pages"][: spare.numel()] = spare
        if op == "tables":
            # (short: the last of the streams that need pages get none)
            free = torch.full((1,), spare.numel(), dtype=torch.int32, device=dev)
            s["free"] = (need.sum(0, keepdim=True) * 3 // 4).clamp_max(free).to(torch.int32) if case["short"] else free
            return s
        take = need.cumsum(0) - need
        j = column - s["held"][:, None]
        new_pages = s["pages"][(take[:, None] + j).clamp(0, total - 1)]
        full = torch.where((j >= 0) & (j < need[:, None]), new_pages, s["table"])
        i = torch.arange(n, device=dev)
        at = s["lens"][:, None] + i
        slots = full.gather(1, (at // page).clamp_max(width - 1).long()).long() * page + at % page
        s["slots"] = torch.where(i < s["new"][:, None], slots, -1).to(torch.int32)
        kv = normal(b, n, 2, case["heads"], case["d"])  # one projection makes keys and values
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        pool = normal(total, 2, page, case["heads"], case["d"])
        s["k_pages"], s["v_pages"] = pool[:, 0], pool[:, 1]
        return s
    if op == "paged":
        b, n, page, hq, hkv, d = (case[k] for k in ("b", "n", "page", "hq", "hkv", "d"))
        lens = _lens(case)
        width = -(-case["longest"] // page)
        held = torch.tensor([-(-x // page) for x in lens], device=dev)
        total = int(sum(-(-x // page) for x in lens)) + 1
        order = shuffled(total)
        column = torch.arange(width, device=dev)
        at = (held.cumsum(0) - held)[:, None] + column
        s["table"] = torch.where(column < held[:, None], order[at.clamp_max(total - 1)], -1).to(torch.int32)
        s["k_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q_lens"] = torch.tensor(_news(case, lens), dtype=torch.int32, device=dev)
        s["q"] = normal(b, n, hq, d)
        pool = normal(total, 2, page, hkv, d)
        s["k_pages"], s["v_pages"] = pool[:, 0], pool[:, 1]
        return s
    b, k, v = case["b"], case["k"], case["v"]
    logits = torch.randn(b, k + 1, v, generator=gen, device=dev) * case["spread"]
    draft = logits[:, :k] + torch.randn(b, k, v, generator=gen, device=dev) * case["noise"]
    s["logits"], s["draft"] = logits.to(_type(case)), draft.to(_type(case))
    # The drafted codes are draws from the draft's probabilities.
    t = max(case["temperature"], 1e-3)
    noise = -(-torch.rand(b, k, v, generator=gen, device=dev, dtype=torch.float64).clamp_min(1e-300).log()).log()
    s["codes"] = (s["draft"].double() / t + noise).argmax(2).to(torch.int32)
    if case["point"]:
        s["draft"] = None
    s["u"] = torch.rand(b, k + 1, generator=gen, device=dev)
    s["n_draft"] = torch.tensor(_drafts(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    form = {"embed": (_embed_plain, _embed_own), "tables": (_tables_plain, _tables_own), "write": (_write_plain, _write_own),
            "paged": (_paged_plain, _paged_own), "verify": (_verify_plain, _verify_own)}
    return form[s["case"]["op"]][bool(own)](s)


def _embed_own(s):
    import haar_wavelet_patching_b200 as hwp
    c = s["case"]
    out = {"y": hwp.embed_codes(s["codes"], s["table"], scale=c["scale"])}
    if c["train"]:
        out["dtable"] = hwp.embed_codes_backward(s["go"], s["codes"], c["v"], scale=c["scale"])
    return out


def _embed_plain(s):
    c = s["case"]
    codes, scale = s["codes"].long(), np.float32(c["scale"]).item()
    out = {"y": (s["table"][codes].float() * scale).to(_type(c))}
    if c["train"]:
        g = torch.zeros(c["v"], c["d"], dtype=torch.float64, device=codes.device)  # (long sums)
        g.index_add_(0, codes, s["go"].double())
        out["dtable"] = (g * scale).to(_type(c))
    return out


def _tables_own(s):
    import haar_wavelet_patching_b200 as hwp
    c = s["case"]
    slots = torch.empty(c["b"], c["n"], dtype=torch.int32, device=s["lens"].device)
    held, free = torch.empty_like(s["held"]), torch.empty_like(s["free"])
    hwp.tok_page_tables(s["lens"], s["new"], s["held"], s["free"], s["pages"], s["table"], slots, held, free, c["page"])
    return {"slots": slots, "table": s["table"], "held": held, "free": free}


def _tables_plain(s):
    c = s["case"]
    page, n, width = c["page"], c["n"], s["table"].shape[1]
    lens, new, held, free = (s[k].long() for k in ("lens", "new", "held", "free"))
    need = ((lens + new + page - 1) // page - held).clamp_min(0)
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= free)
    got = torch.where(served, need, 0)
    j = torch.arange(width, device=lens.device) - held[:, None]
    take = free - 1 - (upto - need)[:, None] - j
    fresh = (j >= 0) & (j < got[:, None])
    table = torch.where(fresh, s["pages"][take.clamp(0, s["pages"].numel() - 1)], s["table"])
    i = torch.arange(n, device=lens.device)
    at = lens[:, None] + i
    slots = table.gather(1, (at // page).clamp_max(width - 1)).long() * page + at % page
    slots = torch.where((i < new[:, None]) & served[:, None], slots, -1)
    return {"slots": slots.to(torch.int32), "table": table, "held": (held + got).to(torch.int32),
            "free": (free - got.sum()).to(torch.int32)}


def _write_own(s):
    import haar_wavelet_patching_b200 as hwp
    hwp.paged_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _write_plain(s):
    c = s["case"]
    slots = s["slots"].flatten().long()
    live = (slots >= 0).nonzero()[:, 0]
    slots = slots[live]
    for x, pages in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
        pages[slots // c["page"], slots % c["page"]] = x.flatten(0, 1)[live]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _paged_own(s):
    import haar_wavelet_patching_b200 as hwp
    return {"o": hwp.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["k_lens"], s["q_lens"])}


def _paged_plain(s):
    c = s["case"]
    b, n, page, hq, hkv, d = (c[k] for k in ("b", "n", "page", "hq", "hkv", "d"))
    width = s["table"].shape[1]
    at = s["table"].clamp_min(0).long()

    def rows(pages):  # [b, hkv, width * page, d]
        return pages[at].view(b, width * page, hkv, d).transpose(1, 2).float()

    q = s["q"].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    p = (q * d ** -0.5) @ rows(s["k_pages"]).transpose(2, 3)
    i = torch.arange(n, device=q.device)
    k_lens, q_lens = s["k_lens"][:, None], s["q_lens"][:, None]
    sees = torch.where(i < q_lens, k_lens - q_lens + i + 1, 0)  # [b, n]
    hidden = torch.arange(width * page, device=q.device) >= sees[:, :, None]
    p = p.view(b, hkv, hq // hkv, n, -1).masked_fill_(hidden[:, None, None], float("-inf"))
    m = p.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)  # (rows without a key)
    p = p.sub_(m).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp_min(1e-30))
    o = p.view(b, hkv, -1, width * page) @ rows(s["v_pages"])
    return {"o": o.view(b, hkv, hq // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d).to(torch.bfloat16)}


def _verify_own(s):
    import haar_wavelet_patching_b200 as hwp
    out, accepted = hwp.verify_codes(s["logits"], s["codes"], s["u"], s["draft"], s["n_draft"],
                                     temperature=s["case"]["temperature"])
    return {"codes": out, "accepted": accepted}


def _probabilities(x, t):
    """In 64 bits: 64,000 borders lie in [0, 1), and a draw next to one has to fall on its right side."""
    if t <= 0:
        return torch.zeros_like(x, dtype=torch.float64).scatter_(2, x.argmax(2, keepdim=True), 1.0)
    x = x.double()
    e = ((x - x.amax(2, keepdim=True)) / np.float32(t).item()).exp_()
    return e.div_(e.sum(2, keepdim=True))


def _verify_plain(s):
    c = s["case"]
    b, k, v = c["b"], c["k"], c["v"]
    t = c["temperature"]
    p = _probabilities(s["logits"], t)
    drafted = s["codes"].long()[..., None]
    q = torch.zeros(b, k, v, dtype=torch.float64, device=p.device).scatter_(2, drafted, 1.0) if s["draft"] is None \
        else _probabilities(s["draft"], t)
    u = s["u"].double()
    yes = u[:, :k] * q.gather(2, drafted)[..., 0] < p[:, :k].gather(2, drafted)[..., 0]
    i = torch.arange(k, device=p.device)
    n_draft = torch.full((b,), k, device=p.device) if s["n_draft"] is None else s["n_draft"].long()
    yes &= i < n_draft[:, None]
    accepted = yes.long().cumprod(1).sum(1)
    row = accepted[:, None, None].expand(b, 1, v)
    p = p.gather(1, row)[:, 0]
    if k:
        r = (p - q.gather(1, row.clamp_max(k - 1))[:, 0]).clamp_min(0.0)
        r = torch.where((accepted < n_draft)[:, None] & (r.sum(1, keepdim=True) > 0), r, p)
    else:
        r = p
    run_ = r.cumsum(1)
    drawn = (run_ <= u[:, k:] * run_[:, -1:]).sum(1).clamp_max(v - 1)
    i = torch.arange(k + 1, device=p.device)
    padded = torch.cat((s["codes"].long(), torch.zeros(b, 1, dtype=torch.long, device=p.device)), 1)
    out = torch.where(i < accepted[:, None], padded, torch.where(i == accepted[:, None], drawn[:, None], -1))
    return {"codes": out.to(torch.int32), "accepted": accepted.to(torch.int32)}


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "embed":
        size = 2 if case["dtype"] == "bf16" else 4
        n, v, d = case["tokens"], case["v"], case["d"]
        rows = n * d * size
        if case["train"]:  # codes, the rows met and the gradient read; y and the table's gradient written
            return {"bytes": 4 * n + (min(n, v) * d + v * d) * size + 2 * rows, "flops": 2 * n * d}
        return {"bytes": 4 * n + min(n, v) * d * size + rows, "flops": n * d}
    if op == "tables":
        return {"bytes": 4 * case["b"] * (case["n"] + 5), "flops": 4 * case["b"] * case["n"]}
    if op == "write":  # (three quarters of the tokens are there)
        n = case["b"] * case["n"]
        return {"bytes": 4 * n + 3 * 2 * n * case["heads"] * case["d"] * 2, "flops": 0}
    if op == "paged":
        n, hq, hkv, d = (case[k] for k in ("n", "hq", "hkv", "d"))
        lens = _lens(case)
        seen = sum(q * x - q * (q - 1) // 2 for q, x in zip(_news(case, lens), lens))
        pages = sum(-(-x // case["page"]) for x in lens)
        return {"bytes": 4 * sum(lens) * hkv * d + 4 * case["b"] * n * hq * d + 4 * pages, "flops": 4 * seen * hq * d}
    size = 2 if case["dtype"] == "bf16" else 4
    rows = sum(_drafts(case)) * (1 if case["point"] else 2) + case["b"]
    return {"bytes": rows * case["v"] * size, "flops": 4 * rows * case["v"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _embed_exact, "tables": _tables_exact, "write": _write_exact, "paged": _paged_exact,
            "verify": _verify_exact}[case["op"]](case, s)


def _embed_exact(case, s):
    """The gradient from the tokens in the order of their codes: differences of a running sum, a slab of channels at a time."""
    scale = float(np.float32(case["scale"]))
    codes = s["codes"].long()
    out = {"y": torch.index_select(s["table"].double() * scale, 0, codes)}
    if case["train"]:
        order = torch.argsort(codes, stable=True)
        ends = torch.searchsorted(codes[order], torch.arange(case["v"], device=codes.device), right=True)
        grad = torch.empty(case["v"], case["d"], dtype=torch.float64, device=codes.device)
        for c0 in range(0, case["d"], 256):
            g = s["go"][order, c0: c0 + 256].double()
            upto = torch.cat((torch.zeros_like(g[:1]), g.cumsum(0)))[ends]
            upto[1:] -= upto[:-1].clone()
            grad[:, c0: c0 + 256] = upto * scale
        once = torch.bincount(codes, minlength=case["v"])
        out["dtable"] = torch.where((once > 0)[:, None], grad, 0.0)
    return out


def _tables_exact(case, s):
    """Stream by stream on the host."""
    lens, new, held, pages, table = (s[k].cpu().tolist() for k in ("lens", "new", "held", "pages", "table"))
    free, page = s["free"].item(), case["page"]
    slots = [[-1] * case["n"] for _ in lens]
    dry = False
    for b, x in enumerate(lens):
        more = max(0, -(-(x + new[b]) // page) - held[b])
        dry = dry or more > free
        if dry and more:
            continue
        for _ in range(more):
            free -= 1
            table[b][held[b]] = pages[free]
            held[b] += 1
        for i in range(new[b]):
            slots[b][i] = table[b][(x + i) // page] * page + (x + i) % page
    return {"slots": torch.tensor(slots, dtype=torch.int32), "table": torch.tensor(table, dtype=torch.int32),
            "held": torch.tensor(held, dtype=torch.int32), "free": torch.tensor([free], dtype=torch.int32)}


def _write_exact(case, s):
    out = {}
    slots = s["slots"].cpu().numpy()
    for name in ("k", "v"):
        flat = s[name + "_pages"].double().flatten(0, 1)
        for b in range(case["b"]):
            n = int((slots[b] >= 0).sum())
            flat[torch.from_numpy(slots[b, :n]).long().to(flat.device)] = s[name][b, :n].double()
        out[name + "_pages"] = flat.view(s[name + "_pages"].shape)
    return out


def _paged_exact(case, s):
    """Stream by stream, head by head and query by query, over the keys that each query sees."""
    b, n, hq, hkv, d = (case[k] for k in ("b", "n", "hq", "hkv", "d"))
    lens = _lens(case)
    news = _news(case, lens)
    o = torch.zeros(b, n, hq, d, dtype=torch.float64, device=s["q"].device)
    for i in range(b):
        if lens[i] == 0:
            continue
        mine = s["table"][i, : -(-lens[i] // case["page"])].long()
        for j in range(hkv):
            heads = slice(j * (hq // hkv), (j + 1) * (hq // hkv))
            k = s["k_pages"][mine, :, j].double().flatten(0, 1)
            v = s["v_pages"][mine, :, j].double().flatten(0, 1)
            for t in range(news[i]):
                m = lens[i] - news[i] + t + 1
                x = torch.einsum("hd,kd->hk", s["q"][i, t, heads].double(), k[:m]) / math.sqrt(d)
                o[i, t, heads] = torch.einsum("hk,kd->hd", torch.softmax(x, 1), v[:m])
    return {"o": o}


def _verify_exact(case, s):
    """Stream by stream on the host, draft by draft until one is refused."""
    k, t = case["k"], float(np.float32(case["temperature"]))
    codes, u = s["codes"].cpu().numpy(), s["u"].double().cpu().numpy()
    drafts = _drafts(case)
    out, accepted = np.full((case["b"], k + 1), -1, dtype=np.int32), np.zeros(case["b"], dtype=np.int32)

    def softmax(x):
        x = x.double().cpu().numpy()
        if t <= 0:
            w = np.zeros(x.shape)
            w[int(np.argmax(x))] = 1.0
            return w
        w = np.exp((x - x.max()) / t)
        return w / w.sum()

    for b in range(case["b"]):
        i = 0
        while True:
            p = softmax(s["logits"][b, i])
            r = p
            if i < drafts[b]:
                x = int(codes[b, i])
                if s["draft"] is None:
                    q = np.zeros(case["v"])
                    q[x] = 1.0
                else:
                    q = softmax(s["draft"][b, i])
                if u[b, i] * q[x] < p[x]:
                    out[b, i] = x
                    i += 1
                    continue
                r = np.maximum(p - q, 0.0)
                r = r if r.sum() > 0 else p
            total = np.cumsum(r)
            out[b, i] = min(int(np.searchsorted(total, u[b, k] * total[-1], side="right")), case["v"] - 1)
            accepted[b] = i
            break
    return {"codes": torch.from_numpy(out), "accepted": torch.from_numpy(accepted)}
