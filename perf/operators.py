"""Cases of the branched-rollout operators: rotary positions with several
axes, the append to a paged cache, and the attention of a batch of branches
over a shared prefix and their own pages.

A world model that answers from one history keeps one prefix (the merged
cache of the past, or the prompt) and continues it in B branches.  A pass of
a layer rotates the new queries and keys by their (time, height, width)
positions, appends the new keys and values to each branch's pages and attends
the prefix together with those pages.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64), or, where `own` is set, with this package's calls.
"""
import math

import torch

own = False

VIDEO = "44,42,42"       # channels turned by time, height and width (D 128)
VIDEO64 = "24,20,20"     # the same for D 64
TEXT = 8                   # branches that add one token each


def listed():
    bf, f32 = "bf16", "f32"
    return [
        # one new token of each of 8 branches: the smallest call, latency counts
        dict(name="rope token b8 h12", op="rope", dtype=bf, H=12, N=TEXT, D=128, dims=VIDEO, halves=False,
             inverse=False, pitch=0, base=10000.0),
        # the queries of a 720p chunk of 3 frames, 40 heads, as the projection leaves them
        dict(name="rope chunk 10800 h40", op="rope", dtype=bf, H=40, N=10800, D=128, dims=VIDEO, halves=False,
             inverse=False, pitch=0, base=10000.0),
        # turning back (the transposed rotation) in 32 bits, rotate-half pairs, an odd count of tokens
        dict(name="rope back 4097 h12 f32", op="rope", dtype=f32, H=12, N=4097, D=64, dims="16,24,24", halves=True,
             inverse=True, pitch=0, base=1000000.0),
        # one token of each of 16 branches, queries turned in the same call
        dict(name="append token b16 h12", op="append", dtype=bf, Hq=12, H=12, B=16, n=1, ragged=False, D=128,
             dims=VIDEO, halves=False, page=64, past=700, fused=True, pad=0),
        # a chunk of 3 frames of 1560 tokens for each of 4 branches
        dict(name="append chunk 4x4680 h12", op="append", dtype=bf, Hq=12, H=12, B=4, n=4680, ragged=False, D=128,
             dims=VIDEO, halves=False, page=128, past=4680, fused=True, pad=0),
        # ragged prompts in 32 bits, unturned queries, rows behind the last branch
        dict(name="append ragged b7 h5 f32", op="append", dtype=f32, Hq=0, H=5, B=7, n=777, ragged=True, D=64,
             dims=VIDEO64, halves=True, page=16, past=333, fused=False, pad=61),
        # one token of each of 4 branches over a short history: latency counts
        dict(name="attend token b4 h12 p2048", op="attend", dtype=bf, Hq=12, H=12, D=128, B=4, n=1, ragged=False,
             C=2048, counts=True, past=300, page=64, block=0, pad=0),
        # one token of each of 16 branches over the merged history of the 40-head model
        dict(name="attend token b16 h40 p11900", op="attend", dtype=bf, Hq=40, H=40, D=128, B=16, n=1, ragged=False,
             C=11900, counts=True, past=1560, page=64, block=0, pad=0),
        # grouped heads, 64 branches of different lengths over a full cache
        dict(name="attend token b64 g5 p32768", op="attend", dtype=bf, Hq=40, H=8, D=128, B=64, n=1, ragged=True,
             C=32768, counts=False, past=2048, page=64, block=0, pad=0),
        # the third chunk of two branches over a full merged cache, frame by frame
        dict(name="attend chunk 2x4680 h12 p32768", op="attend", dtype=bf, Hq=12, H=12, D=128, B=2, n=4680,
             ragged=False, C=32768, counts=True, past=4680, page=128, block=1560, pad=0),
        # ragged prompts of text, token by token, without a prefix, D 64
        dict(name="attend ragged b9 g3 d64", op="attend", dtype=bf, Hq=12, H=4, D=64, B=9, n=601, ragged=True, C=0,
             counts=False, past=257, page=16, block=1, pad=37),
        # 32 bits: a frame of 256 tokens per branch over 1024 merged groups
        dict(name="attend frame 3x256 h4 f32", op="attend", dtype=f32, Hq=4, H=4, D=64, B=3, n=256, ragged=False,
             C=1024, counts=True, past=256, page=32, block=256, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend"))
    D = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    dims = rng.choice((str(D), VIDEO if D == 128 else VIDEO64, f"{D // 2},{D // 4},{D // 4}", f"{D // 4},{D // 4}"))
    halves = rng.random() < 0.5
    if op == "rope":
        H = _log(rng, 1, 40)
        return dict(op=op, dtype=dtype, H=H, N=_log(rng, 1, 400000 // H), D=D, dims=dims, halves=halves,
                    inverse=rng.random() < 0.3, pitch=rng.choice((0, 8, 2 * H * D)), base=10.0 ** rng.randint(3, 6))
    B = _log(rng, 1, 64)
    H = rng.choice((1, 2, 4, 5, 8, 12, 24, 40))
    n = 1 if rng.random() < 0.4 else _log(rng, 1, 60000 // (B * H) + 1)
    ragged = rng.random() < 0.6
    page = rng.choice((16, 32, 64, 128, 256))
    pad = rng.choice((0, 0, rng.randint(1, 50)))
    if op == "append":
        return dict(op=op, dtype=dtype, Hq=H * rng.choice((1, 1, 2)), H=H, B=B, n=n, ragged=ragged, D=D, dims=dims,
                    halves=halves, page=page, past=_log(rng, 1, 4000), fused=rng.random() < 0.6, pad=pad)
    g = rng.choice((1, 1, 2, 3, 5, 8))
    H = min(H, 12)
    n = min(n, max(1, 20000 // (B * H * g)))
    C = 0 if rng.random() < 0.15 else _log(rng, 100, 32768)
    if dtype == "f32":
        C, n = min(C, 4096), min(n, 400)
    return dict(op=op, dtype=dtype, Hq=H * g, H=H, D=D, B=B, n=n, ragged=ragged, C=C, counts=rng.random() < 0.6,
                past=_log(rng, 1, 4000 // max(1, B // 16)), page=page, block=rng.choice((0, 1, 7, 256)), pad=pad)


# ------------------------------------------------------------------- inputs

def _dims(case):
    return [int(d) for d in case["dims"].split(",")]


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _counts(case, salt):
    """New tokens and lengths (new ones included) of each branch: plain
    numbers of the case, so that the work is known without the GPU."""
    u = [((b * 7919 + salt * 104729) % 9973) / 9973.0 for b in range(case["B"])]
    w = [((b * 6007 + salt * 15485863) % 9967) / 9967.0 for b in range(case["B"])]
    new = [case["n"] if not case["ragged"] or case["n"] == 1 else int(x * (case["n"] + 1)) for x in u]
    length = [n + (int(case["past"] * y) if case["ragged"] else case["past"]) for n, y in zip(new, w)]
    return new, length


def _sizes(case):
    """Live rows of each head's prefix: the heads of a merged cache differ."""
    C = case["C"]
    return [C - (h * 997) % (C // 16 + 1) if case["counts"] else C for h in range(case["H"])]


def _freq(case):
    """Radians per position of each pair, axis by axis."""
    base = case.get("base", 10000.0)
    return [base ** (-2.0 * i / d) for d in _dims(case) for i in range(d // 2)]


def _axis(case):
    return [a for a, d in enumerate(_dims(case)) for _ in range(d // 2)]


def _positions(N, axes, g):
    # time steps grow without end, rows and columns of a frame do not
    hi = torch.tensor([100000] + [104] * (axes - 1), device="cuda")
    return (torch.rand(N, axes, generator=g, device="cuda") * hi).to(torch.int32)


def _pages(case, length, g):
    """Pages of every branch, scattered over a pool that has spare ones; what
    nobody wrote holds old values."""
    page, dt = case["page"], _type(case)
    most = max(1, -(-max(length) // page))
    pool = case["B"] * most + 3
    shape = (pool, case["H"], page, case["D"])
    K = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    V = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    order = torch.randperm(pool, generator=g, device="cuda")[: case["B"] * most]
    return K, V, order.view(case["B"], most).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, D = _type(case), case["D"]
    s = dict(case=case)
    if "dims" in case:
        s["freq"] = torch.tensor(_freq(case), dtype=torch.float64, device="cuda")
        s["axis"] = torch.tensor(_axis(case), device="cuda")
    if case["op"] == "rope":
        H, N = case["H"], case["N"]
        rows = torch.randn(N, H * D + case["pitch"], generator=g, device="cuda", dtype=dt)
        s["x"] = rows[:, : H * D].view(N, H, D).transpose(0, 1)     # [H][N][D] as the projection leaves it
        s["pos"] = _positions(N, len(_dims(case)), g)
        s["out"] = torch.zeros(H, N, D, device="cuda", dtype=dt)
        if own:
            import merged_attention_autoregressive_gb300 as m
            s["plan"] = m.RopePlan(D, _dims(case), pairing="halves" if case["halves"] else "adjacent",
                                   freqs=_freq(case))
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    B, H, Hq = case["B"], case["H"], case["Hq"]
    new, length = _counts(case, 1)
    N = max(1, sum(new) + case["pad"])
    s["N"], s["most_new"], s["most"] = N, max(1, max(new)), max(1, max(length))
    cu = [sum(new[:b]) for b in range(B + 1)]
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["len"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    s["K"], s["V"], s["table"] = _pages(case, length, g)
    if case["op"] == "append":
        # queries, keys and values side by side, as one projection leaves them
        rows = torch.randn(N, Hq + 2 * H, D, generator=g, device="cuda", dtype=dt).transpose(0, 1)
        s["q"], s["k"], s["v"] = (rows[:Hq] if case["fused"] else None), rows[Hq:Hq + H], rows[Hq + H:]
        s["pos"] = _positions(N, len(_dims(case)), g)
        s["q_out"] = torch.zeros(Hq, N, D, device="cuda", dtype=dt) if case["fused"] else None
    else:
        s["q"] = (1.5 * torch.randn(Hq, N, D, generator=g, device="cuda")).to(dt)
        s["out"] = torch.zeros(Hq, N, D, device="cuda", dtype=dt)
        s["lse"] = torch.zeros(Hq, N, device="cuda")
        C = case["C"]
        s["size"] = torch.tensor(_sizes(case), dtype=torch.int32, device="cuda")
        s["pK"] = torch.randn(H, C, D, generator=g, device="cuda", dtype=dt)
        s["pV"] = torch.randn(H, C, D, generator=g, device="cuda", dtype=dt)
        # a merged group stands for 1 to 40 keys
        s["m"] = (1 + 40 * torch.rand(H, C, generator=g, device="cuda") ** 4).to(torch.int32)
        s["scale"] = D ** -0.5
    if own:
        import merged_attention_autoregressive_gb300 as m
        s["pages"] = m.PagedKV.view(K=s["K"], V=s["V"], table=s["table"], length=s["len"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "append":
            s["plan"] = m.RopePlan(D, _dims(case), pairing="halves" if case["halves"] else "adjacent",
                                   freqs=_freq(case))
        else:
            s["prefix"] = m.Prefix(s["pK"], s["pV"], m=s["m"] if case["counts"] else None,
                                   size=s["size"]) if case["C"] else None
            s["ws"] = torch.empty(m.branch_workspace_size(Hq, H, N, D), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------- plain forms

def _turn(x, s, pos, sign):
    """x [H][N][D] rotated in 32 bits; the angles of far positions in 64."""
    case = s["case"]
    turned = 2 * s["axis"].numel()
    angle = pos[:, s["axis"]].double() * s["freq"]
    c, n = angle.cos().float(), sign * angle.sin().float()
    y = x.float()
    if case["halves"]:
        a, b = y[..., : turned // 2], y[..., turned // 2: turned]
        r = torch.cat((a * c - b * n, a * n + b * c), -1)
    else:
        a, b = y[..., 0:turned:2], y[..., 1:turned:2]
        r = torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
    return torch.cat((r, y[..., turned:]), -1).to(x.dtype)


def _rows(s):
    """Token ids of each branch [B][most_new], and which of them there are."""
    at = s["cu"][:-1, None].long() + torch.arange(s["most_new"], device="cuda")
    there = at < s["cu"][1:, None]
    return at.clamp(max=s["N"] - 1), there


def _append(s):
    at, there = _rows(s)
    page = s["case"]["page"]
    i = torch.arange(s["most_new"], device="cuda")
    slot = (s["len"] - (s["cu"][1:] - s["cu"][:-1]))[:, None].long() + i
    place = slot[there]
    branch = torch.arange(s["case"]["B"], device="cuda")[:, None].expand_as(there)[there]
    where = s["table"][branch, place // page].long()
    tok = at[there]
    s["K"][where, :, place % page] = _turn(s["k"], s, s["pos"], 1.0)[:, tok].transpose(0, 1)
    s["V"][where, :, place % page] = s["v"][:, tok].transpose(0, 1)
    if not s["case"]["fused"]:
        return s["K"], s["V"]
    s["q_out"][:, tok] = _turn(s["q"], s, s["pos"], 1.0)[:, tok]
    return s["K"], s["V"], s["q_out"]


def _attend(s):
    case = s["case"]
    B, H, Hq, D, C = (case[k] for k in ("B", "H", "Hq", "D", "C"))
    g, n, L = Hq // H, s["most_new"], s["most"]
    at, there = _rows(s)
    q = s["q"][:, at].float().view(H, g, B, n, D).transpose(1, 2)                  # [H][B][g][n][D]
    K = s["K"][s["table"].long()].transpose(2, 3).flatten(1, 2)[:, :L].permute(2, 0, 3, 1).float()
    V = s["V"][s["table"].long()].transpose(2, 3).flatten(1, 2)[:, :L].permute(2, 0, 1, 3).float()
    shared = (q.reshape(H, B * g * n, D) @ s["pK"].float().transpose(1, 2)).view(H, B, g, n, C)
    x = torch.cat((shared, (q.reshape(H, B, g * n, D) @ K).view(H, B, g, n, L)), -1).mul_(s["scale"])
    if case["counts"]:
        x[..., :C] += s["m"].float().log()[:, None, None, None]
    # the token's own place in its branch, and the keys it may see
    place = (s["len"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(n, device="cuda")
    sees = s["len"][:, None].expand(B, n)
    if case["block"]:
        sees = torch.minimum(sees, (place // case["block"] + 1) * case["block"])
    x[..., :C].masked_fill_((torch.arange(C, device="cuda") >= s["size"][:, None])[:, None, None, None], -torch.inf)
    x[..., C:].masked_fill_((torch.arange(L, device="cuda") >= sees[..., None])[None, :, None], -torch.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p[..., :C].reshape(H, B * g * n, C) @ s["pV"].float()).view(H, B, g, n, D)
    o = o + (p[..., C:].reshape(H, B, g * n, L) @ V).view(H, B, g, n, D)
    o = torch.where(total > 0, o / total, 0.0).transpose(1, 2).reshape(Hq, B, n, D)
    lse = (top + total.log()).squeeze(-1).transpose(1, 2).reshape(Hq, B, n)
    s["out"][:, at[there]] = o[:, there].to(s["out"].dtype)
    s["lse"][:, at[there]] = lse[:, there]
    return s["out"], s["lse"]


def run(s):
    case = s["case"]
    if own:
        import merged_attention_autoregressive_gb300 as m
        if case["op"] == "rope":
            m.fastar_rope(s["x"], s["pos"], s["plan"], s["out"], inverse=case["inverse"], status=s["status"])
            return s["out"]
        if case["op"] == "append":
            m.fastar_page_append(s["pages"], s["k"], s["v"], s["cu"], pos=s["pos"], plan=s["plan"], q=s["q"],
                                 q_out=s["q_out"], status=s["status"])
            return (s["K"], s["V"], s["q_out"]) if case["fused"] else (s["K"], s["V"])
        m.fastar_branch_attention(s["q"], s["cu"], s["prefix"], s["pages"], s["scale"], s["out"], lse=s["lse"],
                                  block=case["block"], ws=s["ws"], status=s["status"])
        return s["out"], s["lse"]
    if case["op"] == "rope":
        s["out"].copy_(_turn(s["x"], s, s["pos"], -1.0 if case["inverse"] else 1.0))
        return s["out"]
    return _append(s) if case["op"] == "append" else _attend(s)


# ---------------------------------------------------------------------- work

def _seen(case):
    """(query, key) pairs that are attended over all heads, and the rows of
    the pages that some query sees."""
    new, length = _counts(case, 1)
    pairs, rows, k = 0, 0, case["block"]
    for n, full in zip(new, length):
        past, last = full - n, 0
        if n:
            if k:
                ends = [min(full, ((past + i) // k + 1) * k) for i in range(n)]
                pairs, last = pairs + sum(ends), ends[-1]
            else:
                pairs, last = pairs + n * full, full
        rows += last
    return pairs * case["Hq"], rows


def work(case):
    e, D = (2 if case["dtype"] == "bf16" else 4), case["D"]
    if case["op"] == "rope":
        n = case["N"] * case["H"]
        return {"bytes": 2 * n * D * e + case["N"] * 4 * len(_dims(case)), "flops": 3.0 * n * sum(_dims(case))}
    new, _ = _counts(case, 1)
    N = sum(new)
    if case["op"] == "append":
        heads = 2 * case["H"] + (case["Hq"] if case["fused"] else 0)
        turned = case["H"] + (case["Hq"] if case["fused"] else 0)
        return {"bytes": 2 * N * heads * D * e + N * 4 * len(_dims(case)), "flops": 3.0 * N * turned * sum(_dims(case))}
    pairs, rows = _seen(case)
    size = _sizes(case)
    pairs += N * case["Hq"] // case["H"] * sum(size)
    kv = 2 * D * e * (sum(size) + rows * case["H"]) + (4 * sum(size) if case["counts"] else 0)
    return {"bytes": kv + N * case["Hq"] * (2 * D * e + 4), "flops": 4.0 * D * pairs}


# --------------------------------------------------------------- in 64 bits

def _turned(x, pos, case, sign):
    """x [H][N][D] in 64 bits, as complex numbers times exp(i angle)."""
    ladder, z = [], x.double()
    for a, d in enumerate(_dims(case)):
        f = case.get("base", 10000.0) ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
        ladder.append(pos[:, a, None].double() * f)
    angle = torch.cat(ladder, 1) * sign
    unit = torch.polar(torch.ones_like(angle), angle)
    t = sum(_dims(case))
    if case["halves"]:
        w = torch.complex(z[..., : t // 2].contiguous(), z[..., t // 2: t].contiguous()) * unit
        z = torch.cat((w.real, w.imag, z[..., t:]), -1)
    else:
        w = torch.view_as_complex(z[..., :t].unflatten(-1, (-1, 2)).contiguous()) * unit
        z = torch.cat((torch.view_as_real(w).flatten(-2), z[..., t:]), -1)
    return z


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["x"], s["pos"], case, -1.0 if case["inverse"] else 1.0)
    new, length = _counts(case, 1)
    cu = [sum(new[:b]) for b in range(len(new) + 1)]
    page = case["page"]
    if case["op"] == "append":
        K, V = s["K"].double(), s["V"].double()
        k = _turned(s["k"], s["pos"], case, 1.0)
        for b, (n, full) in enumerate(zip(new, length)):
            for p in range((full - n) // page, -(-full // page)):
                lo, hi = max(full - n, p * page), min(full, (p + 1) * page)
                if hi > lo:
                    t, at = cu[b] + lo - (full - n), int(s["table"][b, p])
                    K[at, :, lo - p * page:hi - p * page] = k[:, t:t + hi - lo]
                    V[at, :, lo - p * page:hi - p * page] = s["v"][:, t:t + hi - lo].double()
        if not case["fused"]:
            return K, V
        q = torch.zeros_like(s["q_out"], dtype=torch.float64)
        q[:, : cu[-1]] = _turned(s["q"], s["pos"], case, 1.0)[:, : cu[-1]]
        return K, V, q
    if work(case)["flops"] > 4e12:
        return None
    H, g, size = case["H"], case["Hq"] // case["H"], _sizes(case)
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    lse = torch.zeros_like(s["lse"], dtype=torch.float64)
    for b, (n, full) in enumerate(zip(new, length)):
        if not n:
            continue
        ids = s["table"][b, : -(-full // page)].long()
        i = torch.arange(full - n, full, device="cuda")
        end = torch.full_like(i, full) if not case["block"] else ((i // case["block"] + 1) * case["block"]).clamp(max=full)
        hidden = torch.arange(full, device="cuda") >= end[:, None]
        for h in range(H):
            k = torch.cat((s["pK"][h, : size[h]], s["K"][ids, h].flatten(0, 1)[:full])).double()
            v = torch.cat((s["pV"][h, : size[h]], s["V"][ids, h].flatten(0, 1)[:full])).double()
            x = s["q"][h * g:(h + 1) * g, cu[b]:cu[b + 1]].double() @ k.T * s["scale"]
            if case["counts"]:
                x[..., : size[h]] += s["m"][h, : size[h]].double().log()
            x[..., size[h]:] = x[..., size[h]:].masked_fill(hidden, -torch.inf)
            out[h * g:(h + 1) * g, cu[b]:cu[b + 1]] = torch.softmax(x, -1) @ v
            lse[h * g:(h + 1) * g, cu[b]:cu[b + 1]] = torch.logsumexp(x, -1)
    return out, lse
