"""Cases of the token-model operators: rotary positions over a (time, height, width) grid,
cross attention to an encoder's states, and sampling of FSQ codes.

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
        # Next-token step of a batch of 16 streams: one token each, at its own place of the grid.
        {"name": "rope_step", "op": "rope_positions", "tokens": 16, "heads": 16, "d": 128, "dt": 44, "dh": 42,
         "dw": 42, "dtype": "bf16", "interleaved": False, "adjoint": False, "row_heads": 16},
        # Queries and keys (32 of the 48 heads of a fused projection) of the 121-frame 704x1280 clip's
        # 16x44x80 latent grid: the largest call of a prompt.
        {"name": "rope_clip", "op": "rope_grid", "t": 16, "h": 44, "w": 80, "heads": 32, "d": 128, "dt": 44,
         "dh": 42, "dw": 42, "dtype": "bf16", "interleaved": False, "adjoint": False, "row_heads": 48},
        # Gradient of a small odd grid in fp32, pairs side by side, part of the head not rotated.
        {"name": "rope_grad_odd", "op": "rope_grid", "t": 7, "h": 33, "w": 45, "heads": 12, "d": 80, "dt": 16,
         "dh": 24, "dw": 24, "dtype": "f32", "interleaved": True, "adjoint": True, "row_heads": 12},
        # Next-token step: 8 streams, each over the encoder states of one 44x80 frame (kept keys and
        # values, ragged), four query heads to a key head.
        {"name": "attn_step", "op": "attn", "b": 8, "nq": 1, "nk": 3520, "hq": 32, "hkv": 8, "d": 128,
         "ragged": True, "empty": False, "train": False},
        # A whole clip's tokens over a 512-long prompt: the largest forward.
        {"name": "attn_clip", "op": "attn", "b": 1, "nq": 56320, "nk": 512, "hq": 16, "hkv": 16, "d": 128,
         "ragged": False, "empty": False, "train": False},
        # Odd lengths, a head size between the tiles' sizes, a padded batch with one clip without a prompt.
        {"name": "attn_odd", "op": "attn", "b": 3, "nq": 1001, "nk": 777, "hq": 12, "hkv": 4, "d": 80,
         "ragged": True, "empty": True, "train": False},
        # Training step of a frame's tokens over another frame's states (3520 x 3520).
        {"name": "attn_train_frame", "op": "attn", "b": 2, "nq": 3520, "nk": 3520, "hq": 16, "hkv": 16, "d": 128,
         "ragged": False, "empty": False, "train": True},
        # Training step of two frames' tokens over padded prompts, shared key heads.
        {"name": "attn_train_text", "op": "attn", "b": 4, "nq": 7040, "nk": 512, "hq": 16, "hkv": 4, "d": 64,
         "ragged": True, "empty": False, "train": True},
        # Next-token step: 4 streams with all filters, each stream with settings of its own.
        {"name": "sample_step", "op": "sample", "rows": 4, "v": CODES, "dtype": "bf16", "temperature": 0.8,
         "top_k": 100, "top_p": 0.95, "min_p": 0.02, "banned": 0, "per_row": True, "spread": 2.5},
        # A batch of streams under nucleus sampling, fp32 logits, a range of codes ruled out.
        {"name": "sample_nucleus", "op": "sample", "rows": 255, "v": CODES, "dtype": "f32", "temperature": 1.0,
         "top_k": 0, "top_p": 0.9, "min_p": 0.0, "banned": 1280, "per_row": False, "spread": 2.0},
        # A quarter of a frame's tokens drawn at once (masked generation).
        {"name": "sample_frame", "op": "sample", "rows": 880, "v": CODES, "dtype": "bf16", "temperature": 0.7,
         "top_k": 500, "top_p": 1.0, "min_p": 0.0, "banned": 0, "per_row": False, "spread": 2.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _axes(rng, d):
    """Even axis widths that together rotate d or somewhat less of d channels."""
    r = d if rng.random() < 0.6 else max(6, d - rng.choice((8, 16)))
    dh = r // 6 * 2
    return {"dt": r // 2 * 2 - 2 * dh, "dh": dh, "dw": dh}


def draw(rng):
    kind = rng.choice(("grid", "grid", "positions", "step", "forward", "forward", "train", "train", "sample", "sample"))
    if kind in ("grid", "positions"):
        d = rng.choice((32, 64, 72, 80, 96, 128))
        heads = rng.randint(1, 32)
        c = {"op": "rope_" + kind, "heads": heads, "d": d, **_axes(rng, d), "dtype": rng.choice(("bf16", "bf16", "f32")),
             "interleaved": rng.random() < 0.5, "adjoint": rng.random() < 0.4,
             "row_heads": heads + rng.choice((0, 0, 1, heads))}
        if kind == "positions":
            return {**c, "tokens": _log(rng, 1, 8192)}
        return {**c, "t": _log(rng, 1, 16), "h": _log(rng, 1, 44), "w": _log(rng, 1, 80)}
    if kind in ("step", "forward", "train"):
        while True:
            hkv, g = rng.randint(1, 16), rng.choice((1, 1, 2, 3, 4, 8))
            c = {"op": "attn", "b": _log(rng, 1, 32 if kind == "step" else 4),
                 "nq": rng.randint(1, 4) if kind == "step" else _log(rng, 1, 20000), "nk": _log(rng, 1, 8192),
                 "hq": hkv * g, "hkv": hkv, "d": rng.choice((32, 64, 64, 80, 96, 128, 128)),
                 "ragged": rng.random() < 0.5, "empty": rng.random() < 0.3, "train": kind == "train"}
            cells = c["b"] * c["hq"] * c["nq"] * c["nk"]
            c["empty"] = c["empty"] and c["b"] > 1
            if cells * (3.5 if kind == "train" else 1.0) * c["d"] <= 16 * 56320 * 512 * 128 \
                    and c["b"] * c["d"] * (hkv * c["nk"] + 2 * c["hq"] * c["nq"]) <= 16 * 56320 * 256:
                return c
    return {"op": "sample", "rows": _log(rng, 1, 800), "v": rng.choice((CODES, CODES, rng.randint(300, 2000), rng.randint(2000, 65000))),
            "dtype": rng.choice(("bf16", "f32")), "temperature": rng.choice((0.0, 0.5, 0.8, 1.0, 1.3)),
            "top_k": rng.choice((0, 0, 1, _log(rng, 2, 4000))), "top_p": rng.choice((1.0, 0.5, 0.9, 0.99)),
            "min_p": rng.choice((0.0, 0.0, 0.05, 0.3)), "banned": rng.choice((0, 0, 100)),
            "per_row": rng.random() < 0.5, "spread": rng.choice((0.5, 1.0, 2.0, 4.0))}


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
ORIGIN = (3, 2, 1)  # the grid's first token is not at the axes' zero: a window of a longer clip
BASES = (10000.0, 10000.0, 10000.0)


def _type(case):
    return torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32


def _dims(case):
    return case["dt"], case["dh"], case["dw"]


def _sizes(case):
    if case["op"] == "rope_positions":
        return 128, 64, 96
    return tuple(n + o for n, o in zip((case["t"], case["h"], case["w"]), ORIGIN))


def _lens(case):
    """Key lengths of a padded batch: full, then shorter and shorter; the last one zero where the case says so."""
    b, nk = case["b"], case["nk"]
    lens = [-(-nk * (b - i) // b) if case["ragged"] else nk for i in range(b)]
    if case["empty"]:
        lens[-1] = 0
    return lens


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev).to(dtype)

    s = {"case": case}
    if case["op"].startswith("rope"):
        tokens = (case["tokens"],) if case["op"] == "rope_positions" else (1, case["t"], case["h"], case["w"])
        rows = normal(*tokens, case["row_heads"], case["d"], dtype=_type(case))
        s["x"] = rows[..., : case["heads"], :]
        sizes = _sizes(case)
        parts = []
        for n, d, base in zip(sizes, _dims(case), BASES):  # [position][pair][cos, sin] of each axis
            freq = base ** (-torch.arange(0, d, 2, dtype=torch.float64, device=dev) / max(d, 1))
            angle = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * freq
            parts.append(torch.stack((angle.cos(), angle.sin()), -1).flatten())
        s["table"] = torch.cat(parts).float()
        if case["op"] == "rope_positions":
            s["pos"] = torch.stack([torch.randint(0, n, tokens, generator=gen, device=dev, dtype=torch.int32)
                                    for n in sizes], -1).contiguous()
        return s
    if case["op"] == "attn":
        b, nq, nk, hq, hkv, d = (case[k] for k in ("b", "nq", "nk", "hq", "hkv", "d"))
        s["q"] = normal(b, nq, hq, d)
        kv = normal(b, nk, 2, hkv, d)  # one projection makes keys and values
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev) if case["ragged"] or case["empty"] else None
        if case["train"]:
            s["go"] = normal(b, nq, hq, d)
        return s
    r, v = case["rows"], case["v"]
    logits = torch.randn(r, v, generator=gen, device=dev) * case["spread"]
    if case["banned"]:
        logits[:, v - min(case["banned"], v - 1):] = float("-inf")
    s["logits"] = logits.to(_type(case))
    s["u"] = torch.rand(r, generator=gen, device=dev)
    s["settings"] = {k: case[k] for k in ("temperature", "top_k", "top_p", "min_p")}
    if case["per_row"]:
        f = 0.75 + 0.5 * torch.rand(r, generator=gen, device=dev)
        s["settings"] = {"temperature": case["temperature"] * f,
                         "top_k": (case["top_k"] * f).to(torch.int32),
                         "top_p": 1 - (1 - case["top_p"]) * f, "min_p": case["min_p"] * f}
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op.startswith("rope"):
        return {"y": _rope_own(s) if own else _rope_plain(s)}
    if op == "attn":
        return _attn_own(s) if own else _attn_plain(s)
    return _sample_own(s) if own else _sample_plain(s)


def _rope_own(s):
    import haar_wavelet_patching_b200 as hwp
    c = s["case"]
    if c["op"] == "rope_positions":
        f = hwp.rope_positions_adjoint if c["adjoint"] else hwp.rope_positions
        return f(s["x"], s["pos"], s["table"], _sizes(c), _dims(c), interleaved=c["interleaved"])
    f = hwp.rope_grid_adjoint if c["adjoint"] else hwp.rope_grid
    return f(s["x"], s["table"], _sizes(c), _dims(c), origin=ORIGIN, interleaved=c["interleaved"])


def _rope_plain(s):
    c, x, table = s["case"], s["x"], s["table"]
    sizes, dims = _sizes(c), _dims(c)
    nt, nh, nw = (n * d for n, d in zip(sizes, dims))
    tt, th, tw = (p.view(n, d // 2, 2) for p, n, d in zip(table.split((nt, nh, nw)), sizes, dims))
    if c["op"] == "rope_positions":
        p = s["pos"].long()
        cs = torch.cat((tt[p[:, 0]], th[p[:, 1]], tw[p[:, 2]]), 1)
    else:
        t, h, w = c["t"], c["h"], c["w"]
        shape = (t, h, w, -1, 2)
        cs = torch.cat((tt[ORIGIN[0]:, None, None].expand(*shape), th[None, ORIGIN[1]:, None].expand(*shape),
                        tw[None, None, ORIGIN[2]:].expand(*shape)), 3)
    cos, sin = cs[..., None, :, 0], cs[..., None, :, 1]
    if c["adjoint"]:
        sin = -sin
    r = sum(dims)
    f = x.float()
    a, b = (f[..., 0:r:2], f[..., 1:r:2]) if c["interleaved"] else (f[..., : r // 2], f[..., r // 2: r])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((ya, yb), -1).flatten(-2) if c["interleaved"] else torch.cat((ya, yb), -1)
    return torch.cat((y, f[..., r:]), -1).to(x.dtype)


def _attn_own(s):
    import haar_wavelet_patching_b200 as hwp
    if not s["case"]["train"]:
        return {"o": hwp.cross_attention(s["q"], s["k"], s["v"], s["lens"])}
    o, lse = hwp.cross_attention(s["q"], s["k"], s["v"], s["lens"], with_lse=True)
    dq, dk, dv = hwp.cross_attention_backward(s["q"], s["k"], s["v"], o, lse, s["go"], s["lens"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _attn_plain(s):
    c = s["case"]
    b, nq, nk, hq, hkv, d = (c[k] for k in ("b", "nq", "nk", "hq", "hkv", "d"))
    scale = d ** -0.5

    def rows(x):  # [b, nq, hq, d] -> [b, hkv, group * nq, d]
        return x.float().transpose(1, 2).reshape(b, hkv, -1, d)

    def back(x, n, heads):
        return x.reshape(b, heads, n, d).transpose(1, 2).to(torch.bfloat16)

    q, k, v = rows(s["q"]), s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    p = (q * scale) @ k.transpose(2, 3)
    if s["lens"] is not None:
        p.masked_fill_((torch.arange(nk, device=q.device) >= s["lens"][:, None])[:, None, None], float("-inf"))
    m = p.amax(3, keepdim=True)
    m0 = m.clamp_min(torch.finfo(torch.float32).min)  # rows without a key
    p = p.sub_(m0).exp_()
    z = p.sum(3, keepdim=True)
    p = p.div_(z.clamp_min(1e-30))
    o = p @ v
    out = {"o": back(o, nq, hq)}
    if not c["train"]:
        return out
    out["lse"] = (m + z.log()).view(b, hq, nq)
    go = rows(s["go"])
    out["dv"] = back(p.transpose(2, 3) @ go, nk, hkv)
    ds = (go @ v.transpose(2, 3)).sub_((go * o).sum(3, keepdim=True)).mul_(p).mul_(scale)
    out["dq"] = back(ds @ k, nq, hq)
    out["dk"] = back(ds.transpose(2, 3) @ q, nk, hkv)
    return out


def _sample_own(s):
    import haar_wavelet_patching_b200 as hwp
    idx, logprob = hwp.sample_codes(s["logits"], s["u"], with_logprob=True, **s["settings"])
    return {"idx": idx, "logprob": logprob}


def _sample_plain(s):
    """In 64 bits: 64,000 borders lie in [0, 1), and a draw next to one has to fall on its right side."""
    g = s["settings"]
    r, v = s["logits"].shape

    def column(x):
        x = x if torch.is_tensor(x) else torch.full((r,), x, device=s["u"].device, dtype=torch.float32)
        return x.double()[:, None]

    t, top_k, top_p, min_p = (column(g[k]) for k in ("temperature", "top_k", "top_p", "min_p"))
    x = s["logits"].double()
    x, order = torch.sort(x, dim=1, descending=True, stable=True)  # ties: the lower index first
    z = (x - x[:, :1]) / t.clamp_min(1e-300)
    z = torch.where(x == x[:, :1], 0.0, z)
    rank = torch.arange(v, device=x.device)
    keep = (rank < torch.where(t <= 0, 1.0, torch.where(top_k <= 0, float(v), top_k))) & (z > float("-inf"))
    e = z.exp() * keep
    before = e.cumsum(1) - e
    keep &= (top_p >= 1) | (before < top_p * e.sum(1, keepdim=True)) | (rank == 0)
    keep &= e >= min_p.clamp_max(1.0)
    e = torch.zeros_like(e).scatter_(1, order, e * keep)  # kept weights, by index
    cum = e.cumsum(1)
    total = cum[:, -1:]
    idx = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    chosen = e.gather(1, idx.clamp_max(v - 1))
    return {"idx": idx[:, 0].to(torch.int32), "logprob": (chosen / total).log()[:, 0].float()}


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def work(case):
    if case["op"].startswith("rope"):
        n = case["tokens"] if case["op"] == "rope_positions" else case["t"] * case["h"] * case["w"]
        size = 2 if case["dtype"] == "bf16" else 4
        table = sum(a * b for a, b in zip(_sizes(case), _dims(case))) * 4
        if case["op"] == "rope_positions":
            table = min(table, n * sum(_dims(case)) * 4) + 12 * n
        return {"bytes": 2 * n * case["heads"] * case["d"] * size + table, "flops": 3 * n * case["heads"] * sum(_dims(case))}
    if case["op"] == "attn":
        b, nq, hq, hkv, d = (case[k] for k in ("b", "nq", "hq", "hkv", "d"))
        keys = sum(_lens(case))
        q, kv = 2 * b * nq * hq * d, 2 * 2 * keys * hkv * d
        if case["train"]:  # q, k, v, go read; o, lse, dq, dk, dv written
            return {"bytes": 4 * q + 2 * kv + 4 * b * nq * hq, "flops": 14 * keys * nq * hq * d}
        return {"bytes": 2 * q + kv, "flops": 4 * keys * nq * hq * d}
    n = case["rows"] * case["v"]
    return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 12 * case["rows"], "flops": 4 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rope"):
        return {"y": _rope_exact(case, s)}
    if case["op"] == "attn":
        return _attn_exact(case, s)
    if case["rows"] * case["v"] > 20e6:
        return None
    return _sample_exact(case, s)


def _rope_exact(case, s):
    """Each pair as a complex number, turned by its angle."""
    x = s["x"].double()
    dims, sizes = _dims(case), _sizes(case)
    if case["op"] == "rope_positions":
        pos = [s["pos"][:, a].double() for a in range(3)]
    else:
        n = (case["t"], case["h"], case["w"])
        grids = torch.meshgrid(*(torch.arange(m, device=x.device) + o for m, o in zip(n, ORIGIN)), indexing="ij")
        pos = [g.double() for g in grids]
    assert all(float(p.max()) < n for p, n in zip(pos, sizes))
    angles = []
    for a in range(3):
        for i in range(dims[a] // 2):
            angles.append(pos[a] * BASES[a] ** (-2.0 * i / dims[a]))
    half = len(angles)
    y = x.clone()
    for i, angle in enumerate(angles):
        turn = torch.polar(torch.ones_like(angle), -angle if case["adjoint"] else angle)[..., None]
        ca, cb = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        out = torch.complex(x[..., ca], x[..., cb]) * turn
        y[..., ca], y[..., cb] = out.real, out.imag
    return y


def _attn_exact(case, s):
    """Head by head, over the keys that each batch entry has."""
    b, nq, nk, hq, hkv, d = (case[k] for k in ("b", "nq", "nk", "hq", "hkv", "d"))
    lens = _lens(case)
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=s["q"].device)  # noqa: E731
    o, lse = new(b, nq, hq, d), new(b, hq, nq)
    dq, dk, dv = (new(b, nq, hq, d), new(b, nk, hkv, d), new(b, nk, hkv, d)) if case["train"] else (None,) * 3
    for i in range(b):
        for h in range(hq):
            j, n = h // (hq // hkv), lens[i]
            if n == 0:
                lse[i, h] = float("-inf")
                continue
            q, k, v = s["q"][i, :, h].double(), s["k"][i, :n, j].double(), s["v"][i, :n, j].double()
            x = torch.einsum("qd,kd->qk", q, k) / math.sqrt(d)
            lse[i, h] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[i, h][:, None])
            o[i, :, h] = torch.einsum("qk,kd->qd", p, v)
            if case["train"]:
                g = s["go"][i, :, h].double()
                dv[i, :n, j] += torch.einsum("qk,qd->kd", p, g)
                dp = torch.einsum("qd,kd->qk", g, v)
                dx = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                dq[i, :, h] = torch.einsum("qk,kd->qd", dx, k)
                dk[i, :n, j] += torch.einsum("qk,qd->kd", dx, q)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if case["train"] else {"o": o}


def _sample_exact(case, s):
    """Row by row on the host."""
    logits = s["logits"].double().cpu().numpy()
    u = s["u"].double().cpu().numpy()
    g = {k: (x.double().cpu().numpy() if torch.is_tensor(x) else np.full(len(u), np.float32(x), dtype=np.float64))
         for k, x in s["settings"].items()}
    idx, logprob = np.zeros(len(u), dtype=np.int32), np.zeros(len(u))
    for i, x in enumerate(logits):
        if g["temperature"][i] <= 0:
            idx[i] = np.argmax(x)
            continue
        order = np.argsort(-x, kind="stable")
        order = order[np.isfinite(x[order])]
        if g["top_k"][i] > 0:
            order = order[: int(g["top_k"][i])]
        w = np.exp((x[order] - x[order[0]]) / g["temperature"][i])
        if g["top_p"][i] < 1:
            n = max(1, int(np.searchsorted(np.cumsum(w), g["top_p"][i] * w.sum(), side="left")) + 1)
            order, w = order[:n], w[:n]
        live = w >= min(g["min_p"][i], 1.0)
        order, w = order[live], w[live]
        by = np.argsort(order)
        order, w = order[by], w[by]
        c = np.cumsum(w)
        n = min(int(np.searchsorted(c, u[i] * c[-1], side="right")), len(c) - 1)
        idx[i], logprob[i] = order[n], math.log(w[n] / c[-1])
    return {"idx": torch.from_numpy(idx), "logprob": torch.from_numpy(logprob)}
