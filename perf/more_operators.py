"""Cases of the operators that draft tokens for branched rollouts and bound
their pages: attention of a tree of drafted tokens over a shared prefix and
pages, the packing of the drafts that were accepted, the attention weight that
every cached row has drawn, and the eviction of the rows that drew least.

A rollout that drafts adds a small tree of tokens to each branch, attends them
all at once, keeps one path of the tree, and adds the weights of what it kept to
the masses of the cached rows.  When a branch holds more rows than its budget,
each head drops those that drew the least attention.

`run` computes an operator in its plain form (elementary torch operations in
32 bits), or, where `own` is set, with this package's calls.
"""
import math

import torch

own = False


def listed():
    bf, f32 = "bf16", "f32"
    return [
        # a binary tree of 15 drafts for each of 4 branches over a short history: latency counts
        dict(name="tree b4 n15 h12 p2048", op="tree", dtype=bf, Hq=12, H=12, D=128, B=4, n=15, ragged=False, binary=True,
             C=2048, counts=True, past=300, page=64, pad=0),
        # 31 drafts for each of 16 branches over the merged history of the 40-head model
        dict(name="tree b16 n31 h40 p11900", op="tree", dtype=bf, Hq=40, H=40, D=128, B=16, n=31, ragged=False,
             binary=False, C=11900, counts=True, past=1560, page=64, pad=0),
        # grouped heads, trees and histories of different sizes over a full cache, padding behind
        dict(name="tree b32 n64 g5 p32768", op="tree", dtype=bf, Hq=40, H=8, D=128, B=32, n=64, ragged=True,
             binary=False, C=32768, counts=False, past=2048, page=64, pad=29),
        # 32 bits, D 64
        dict(name="tree b3 n63 h4 f32", op="tree", dtype=f32, Hq=4, H=4, D=64, B=3, n=63, ragged=False, binary=True,
             C=1024, counts=True, past=256, page=32, pad=0),
        # the accepted path of 31 drafts of 16 branches: latency counts
        dict(name="keep b16 31to6 h12", op="keep", dtype=bf, H=12, D=128, B=16, n=31, keep=6, ragged=False, past=1560,
             page=64),
        # half of the tokens of a chunk of 3 frames stay in each of 4 branches
        dict(name="keep b4 4680to2340 h12", op="keep", dtype=bf, H=12, D=128, B=4, n=4680, keep=2340, ragged=False,
             past=4680, page=128),
        # one token of each of 16 branches over a full budget, 40 heads
        dict(name="mass token b16 h40", op="mass", dtype=bf, Hq=40, H=40, D=128, B=16, n=1, ragged=False, past=4680,
             page=64, block=0, rows=False, decay=1.0, pad=0),
        # a chunk of 3 frames for each of 2 branches, frame by frame
        dict(name="mass chunk 2x4680 h12", op="mass", dtype=bf, Hq=12, H=12, D=128, B=2, n=4680, ragged=False, past=4680,
             page=128, block=1560, rows=False, decay=1.0, pad=0),
        # accepted drafts of ragged branches in 32 bits, grouped heads, old weights fade
        dict(name="mass drafts b9 g3 f32", op="mass", dtype=f32, Hq=12, H=4, D=64, B=9, n=24, ragged=True, past=1200,
             page=16, block=1, rows=True, decay=0.9, pad=7),
        # one row over the budget in each of 16 branches: latency counts
        dict(name="evict step b16 h12", op="evict", dtype=bf, H=12, D=128, B=16, L=1561, ragged=False, budget=1560,
             first=4, recent=256, page=64, born=True),
        # a frame of 1560 tokens over the budget of three, 40 heads
        dict(name="evict frame b4 h40", op="evict", dtype=bf, H=40, D=128, B=4, L=6240, ragged=False, budget=4680,
             first=16, recent=1600, page=128, born=True),
        # long prompts of different lengths down to 8192 rows, once, so that positions tell the age; 32 bits
        dict(name="evict prompt b4 h8 f32", op="evict", dtype=f32, H=8, D=64, B=4, L=32768, ragged=True, budget=8192,
             first=0, recent=1024, page=256, born=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tree", "tree", "keep", "mass", "mass", "evict"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    D = rng.choice((64, 128))
    B, H = _log(rng, 1, 48), rng.choice((1, 2, 4, 5, 8, 12, 40))
    page = rng.choice((16, 32, 64, 128, 256))
    ragged = rng.random() < 0.6
    g = rng.choice((1, 1, 2, 3, 5, 8))
    if op == "tree":
        H, f32 = min(H, 12), dtype == "f32"
        C = 0 if rng.random() < 0.15 else _log(rng, 100, 4096 if f32 else 32768)
        n = _log(rng, 1, min(200, max(1, (6000 if f32 else 20000) // (B * H * g))))
        return dict(op=op, dtype=dtype, Hq=H * g, H=H, D=D, B=B, n=n, ragged=ragged, binary=rng.random() < 0.3, C=C,
                    counts=rng.random() < 0.6, past=_log(rng, 1, 4000 // max(1, B // 16)), page=page,
                    pad=rng.choice((0, 0, rng.randint(1, 50))))
    if op == "keep":
        n = _log(rng, 1, 200000 // (B * H) + 1)
        return dict(op=op, dtype=dtype, H=H, D=D, B=B, n=n, keep=rng.randint(0, n), ragged=ragged,
                    past=_log(rng, 1, 4000), page=page)
    if op == "mass":
        H = min(H, 12)
        n = 1 if rng.random() < 0.4 else _log(rng, 1, (6000 if dtype == "f32" else 40000) // (B * H * g) + 1)
        return dict(op=op, dtype=dtype, Hq=H * g, H=H, D=D, B=B, n=n, ragged=ragged,
                    past=_log(rng, 1, 5000 // max(1, B // 8)), page=page, block=rng.choice((0, 1, 7, 256)),
                    rows=rng.random() < 0.3, decay=rng.choice((1.0, 1.0, 0.95)), pad=rng.choice((0, 0, rng.randint(1, 50))))
    L = _log(rng, 1, min(32768, 600000 // (B * H) + 1))
    budget = rng.randint(0, L + L // 8)
    first = rng.randint(0, min(16, budget))
    return dict(op=op, dtype=dtype, H=H, D=D, B=B, L=L, ragged=ragged, budget=budget, first=first,
                recent=rng.randint(0, (budget - first) // 2), page=page, born=rng.random() < 0.7)


# ------------------------------------------------------------------- inputs

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _u(b, salt):
    return ((b * 7919 + salt * 104729) % 9973) / 9973.0


def _counts(case):
    """New tokens and lengths (new ones included) of each branch: plain
    numbers of the case, so that the work is known without the GPU."""
    n, B = case["n"], case["B"]
    new = [n if not case["ragged"] or n == 1 else int(_u(b, 1) * (n + 1)) for b in range(B)]
    return new, [m + (int(case["past"] * _u(b, 5)) if case["ragged"] else case["past"]) for b, m in enumerate(new)]


def _parents(case, new):
    """The tree of each branch: token i hangs on an earlier token, or on the
    last cached one (-1)."""
    def parent(b, i):
        return (i + 1) // 2 - 1 if case["binary"] else int(_u(b * 977 + i, 3) * (i + 1)) - 1
    return [[parent(b, i) for i in range(n)] for b, n in enumerate(new)]


def _kept(case, new):
    """Ascending numbers of the tokens that stay, branch after branch."""
    kept = []
    for b, n in enumerate(new):
        k = min(case["keep"], n)
        if case["ragged"]:
            k = min(n, int(_u(b, 7) * (2 * k + 1)))
        kept.append([(2 * j * n + n) // (2 * k) for j in range(k)])
    return kept


def _lengths(case):
    return [case["L"] if not case["ragged"] else int(_u(b, 9) * (case["L"] + 1)) for b in range(case["B"])]


def _sizes(case):
    """Live rows of each head's prefix: the heads of a merged cache differ."""
    C = case["C"]
    return [C - (h * 997) % (C // 16 + 1) if case["counts"] else C for h in range(case["H"])]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


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
    dt, D, B, H, op = _type(case), case["D"], case["B"], case["H"], case["op"]
    s = dict(case=case, scale=D ** -0.5)
    if op == "evict":
        new, length = [], _lengths(case)
    else:
        new, length = _counts(case)
        s["cu"], s["most_new"] = _ints(_offsets(new)), max(1, max(new))
    s["len"], s["most"] = _ints(length), max(1, max(length))
    s["K"], s["V"], s["table"] = _pages(case, length, g)
    pool, page = s["K"].shape[0], case["page"]
    if op == "keep":
        kept = _kept(case, new)
        cu = _offsets(new)
        s["rows"] = _ints([cu[b] + i for b, k in enumerate(kept) for i in k])
        s["cu_keep"] = _ints(_offsets([len(k) for k in kept]))
    if op in ("tree", "mass"):
        Hq, N = case["Hq"], max(1, sum(new) + case["pad"])
        s["N"] = N
        s["q"] = (1.5 * torch.randn(Hq, N, D, generator=g, device="cuda")).to(dt)
    if op == "tree":
        s["parent"] = _ints([p for t in _parents(case, new) for p in t] + [-1] * (s["N"] - sum(new)))
        s["out"] = torch.zeros(Hq, s["N"], D, device="cuda", dtype=dt)
        s["lse"] = torch.zeros(Hq, s["N"], device="cuda")
        C = case["C"]
        s["size"] = _ints(_sizes(case))
        s["pK"] = torch.randn(H, C, D, generator=g, device="cuda", dtype=dt)
        s["pV"] = torch.randn(H, C, D, generator=g, device="cuda", dtype=dt)
        # a merged group stands for 1 to 40 keys
        s["m"] = (1 + 40 * torch.rand(H, C, generator=g, device="cuda") ** 4).to(torch.int32)
    if op in ("mass", "evict"):
        # what the rows have drawn so far: a few draw most of it
        s["mass"] = 40 * torch.rand(pool, H, page, generator=g, device="cuda") ** 6
        s["born"], s["total"] = torch.zeros(pool, H, page, dtype=torch.int32, device="cuda"), s["len"] + 500
    if op == "mass":
        # tokens that were taken out of a longer list (the drafts that were accepted), or all of them
        s["take"] = torch.randperm(s["N"], generator=g, device="cuda")[: sum(new)].sort().values.to(torch.int32)
        if not case["rows"]:
            s["take"] = torch.arange(sum(new), dtype=torch.int32, device="cuda")
        # the log-sum-exp of scores of normal keys, a prefix of as many keys beside
        keys = torch.tensor([2.0 * x + 1 for n, x in zip(new, length) for _ in range(n)], device="cuda").log()
        s["lse"] = torch.zeros(Hq, s["N"], device="cuda")
        s["lse"][:, s["take"].long()] = keys
        s["lse"] += s["q"].float().square().sum(-1) * (s["scale"] ** 2 / 2)
    if op == "evict":
        # tokens of earlier evictions lie anywhere, the last eighth in their order
        p = torch.arange(s["most"], device="cuda")
        old = (s["len"] - s["len"] // 8)[:, None, None].expand(B, H, 1)
        shuffled = torch.rand(B, H, s["most"], generator=g, device="cuda").masked_fill(p >= old, 2.0).argsort(-1)
        number = torch.where(p < old, shuffled, p)
        number = torch.where(number < 20, number, number + 500).to(torch.int32)
        page_of, at = s["table"].long()[:, p // page], p % page
        s["born"][page_of[:, None], torch.arange(H, device="cuda")[:, None], at] = number
        s["out_mass"], s["out_born"] = torch.zeros_like(s["mass"]), torch.zeros_like(s["born"])
    if own:
        import merged_attention_autoregressive_gb300 as m
        s["pages"] = m.PagedKV.view(K=s["K"], V=s["V"], table=s["table"], length=s["len"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op == "tree":
            s["prefix"] = m.Prefix(s["pK"], s["pV"], m=s["m"] if case["counts"] else None,
                                   size=s["size"]) if case["C"] else None
            s["ws"] = torch.empty(m.branch_workspace_size(case["Hq"], H, s["N"], D), dtype=torch.uint8, device="cuda")
        if op == "mass":
            s["held"] = m.PageMass.view(s["mass"], s["born"], s["total"])
            s["ws"] = torch.empty(max(1, m.mass_workspace_size(case["Hq"], H, s["take"].numel(), D)), dtype=torch.uint8,
                                  device="cuda")
        if op == "evict":
            born = case["born"]
            s["held"] = m.PageMass.view(s["mass"], s["born"] if born else None, s["total"] if born else None)
            s["held_out"] = m.PageMass.view(s["out_mass"], s["out_born"] if born else None, s["total"] if born else None)
    return s


# --------------------------------------------------------------- plain forms

def _rows(s, count):
    """Token ids of each branch [B][most_new], and which of them there are."""
    at = s["cu"][:-1, None].long() + torch.arange(s["most_new"], device="cuda")
    there = at < s["cu"][1:, None]
    return at.clamp(max=max(0, count - 1)), there


def _keys(s):
    """The rows of every branch in 32 bits, [H][B][L][D]."""
    return [x[s["table"].long()].transpose(2, 3).flatten(1, 2)[:, : s["most"]].permute(2, 0, 1, 3).float()
            for x in (s["K"], s["V"])]


def _closure(parent, n):
    """Whether token j is token i or one of those above it: [B][n][n]."""
    reach = torch.eye(n, device="cuda") + (parent[..., None] == torch.arange(n, device="cuda")).float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = ((reach @ reach) > 0).float()
    return reach > 0


def _tree(s):
    case = s["case"]
    B, H, Hq, D, C = (case[k] for k in ("B", "H", "Hq", "D", "C"))
    g, n, L = Hq // H, s["most_new"], s["most"]
    at, there = _rows(s, s["N"])
    q = s["q"][:, at].float().view(H, g, B, n, D).transpose(1, 2)                  # [H][B][g][n][D]
    K, V = _keys(s)
    shared = (q.reshape(H, B * g * n, D) @ s["pK"].float().transpose(1, 2)).view(H, B, g, n, C)
    x = torch.cat((shared, (q.reshape(H, B, g * n, D) @ K.transpose(2, 3)).view(H, B, g, n, L)), -1).mul_(s["scale"])
    if case["counts"]:
        x[..., :C] += s["m"].float().log()[:, None, None, None]
    # positions before the drafts, and the drafts above a token
    past = s["len"] - (s["cu"][1:] - s["cu"][:-1])
    draft = torch.arange(L, device="cuda") - past[:, None]                          # [B][L]
    above = _closure(torch.where(there, s["parent"][at], -1), n)
    above = above.gather(2, draft.clamp(0, n - 1)[:, None].expand(B, n, L)) & (draft < n)[:, None]
    sees = torch.where((draft < 0)[:, None], True, above)                           # [B][n][L]
    x[..., :C].masked_fill_((torch.arange(C, device="cuda") >= s["size"][:, None])[:, None, None, None], -torch.inf)
    x[..., C:].masked_fill_(~sees[None, :, None], -torch.inf)
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


def _keep(s):
    page = s["case"]["page"]
    i = torch.arange(s["rows"].numel(), device="cuda")
    b = torch.searchsorted(s["cu_keep"][1:].long(), i, right=True)
    past = s["len"] - (s["cu"][1:] - s["cu"][:-1])
    old, new = past[b] + s["rows"] - s["cu"][b], past[b] + i - s["cu_keep"][b]
    old_page, new_page = s["table"][b, old // page].long(), s["table"][b, new // page].long()
    s["K"][new_page, :, new % page] = s["K"][old_page, :, old % page]
    s["V"][new_page, :, new % page] = s["V"][old_page, :, old % page]
    return s["K"], s["V"]


def _mass(s):
    case = s["case"]
    B, H, Hq, D, page = (case[k] for k in ("B", "H", "Hq", "D", "page"))
    g, n, L = Hq // H, s["most_new"], s["most"]
    at, there = _rows(s, s["take"].numel())
    row = s["take"][at].long() if s["take"].numel() else at
    q = s["q"][:, row].float().view(H, g, B, n, D).transpose(1, 2).reshape(H, B, g * n, D)
    lse = s["lse"][:, row].view(H, g, B, n).transpose(1, 2)
    count = s["cu"][1:] - s["cu"][:-1]
    past = s["len"] - count
    place = past[:, None] + torch.arange(n, device="cuda")
    sees = s["len"][:, None].expand(B, n)
    if case["block"]:
        sees = torch.minimum(sees, (place // case["block"] + 1) * case["block"])
    sees = torch.where(there, sees, 0)
    p = torch.arange(L, device="cuda")
    w = (q @ _keys(s)[0].transpose(2, 3)).view(H, B, g, n, L).mul_(s["scale"]).sub_(lse[..., None]).exp_()
    drawn = w.masked_fill_((p >= sees[..., None])[None, :, None], 0.0).flatten(2, 3).sum(2).transpose(0, 1)  # [B][H][L]
    live = (p < s["len"][:, None]) & (count > 0)[:, None]                          # [B][L]
    page_of, at = s["table"].long()[:, p // page], p % page
    fresh = p >= past[:, None]
    old = torch.where(fresh[:, None], 0.0, case["decay"] * s["mass"][page_of[:, None], torch.arange(H, device="cuda")[:, None], at])
    branch, where = live.nonzero(as_tuple=True)
    s["mass"][page_of[branch, where], :, at[where]] = (old + drawn).transpose(1, 2)[branch, where]
    branch, where = (live & fresh).nonzero(as_tuple=True)
    number = s["total"][branch] - s["len"][branch] + where
    s["born"][page_of[branch, where], :, at[where]] = number[:, None].expand(-1, H).to(torch.int32)
    return s["mass"], s["born"]


def _evict(s):
    case = s["case"]
    B, H, page, budget, first, recent = (case[k] for k in ("B", "H", "page", "budget", "first", "recent"))
    L = s["most"]
    p, head = torch.arange(L, device="cuda"), torch.arange(H, device="cuda")[:, None]
    page_of, at = s["table"].long()[:, None, p // page], p % page                  # [B][1][L]
    mass, born = s["mass"][page_of, head, at], s["born"][page_of, head, at]        # [B][H][L]
    live = (p < s["len"][:, None])[:, None]
    age, total = (born, s["total"]) if case["born"] else (p.expand(B, H, L), s["len"])
    safe = (age < first) | (age >= total[:, None, None] - recent)
    value = torch.where(safe, torch.inf, mass).masked_fill(~live, -torch.inf)
    order = value.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(B, H, L, dtype=torch.bool, device="cuda").scatter_(-1, order[..., :budget], True) & live
    # kept rows from the budget on go into the holes before it, in order
    hole, mover = (~kept & live)[..., :budget], kept[..., budget:]
    nth = mover.cumsum(-1) - 1
    holes = hole.to(torch.int8).argsort(dim=-1, descending=True, stable=True)       # the holes in order, then the rest
    b, h, j = mover.nonzero(as_tuple=True)
    old, new = budget + j, holes[b, h, nth[b, h, j]] if budget else j
    old_page, new_page = s["table"][b, old // page].long(), s["table"][b, new // page].long()
    s["K"][new_page, h, new % page] = s["K"][old_page, h, old % page]
    s["V"][new_page, h, new % page] = s["V"][old_page, h, old % page]
    moves = [(s["mass"], s["out_mass"])] + ([(s["born"], s["out_born"])] if case["born"] else [])
    stay = kept & (p < budget)
    sb, sh, sp = stay.nonzero(as_tuple=True)
    src_page = s["table"][sb, sp // page].long()

    def carry(x, y):
        y[src_page, sh, sp % page] = x[src_page, sh, sp % page]
        y[new_page, h, new % page] = x[old_page, h, old % page]
        return y

    return (s["K"], s["V"], *(carry(x, y) for x, y in moves))


def run(s):
    op = s["case"]["op"]
    if own:
        import merged_attention_autoregressive_gb300 as m
        case = s["case"]
        if op == "tree":
            m.fastar_tree_attention(s["q"], s["cu"], s["parent"], s["prefix"], s["pages"], s["scale"], s["out"],
                                    lse=s["lse"], ws=s["ws"], status=s["status"])
            return s["out"], s["lse"]
        if op == "keep":
            m.fastar_page_keep(s["pages"], s["cu"], s["rows"], s["cu_keep"], status=s["status"])
            return s["K"], s["V"]
        if op == "mass":
            m.fastar_page_mass(s["pages"], s["q"], s["lse"], s["cu"], s["scale"], s["held"], block=case["block"],
                               rows=s["take"] if case["rows"] else None, decay=case["decay"], ws=s["ws"],
                               status=s["status"])
            return s["mass"], s["born"]
        m.fastar_page_evict(s["pages"], s["held"], case["budget"], first=case["first"], recent=case["recent"],
                            out=s["held_out"], status=s["status"])
        return (s["K"], s["V"], s["out_mass"], s["out_born"]) if case["born"] else (s["K"], s["V"], s["out_mass"])
    return {"tree": _tree, "keep": _keep, "mass": _mass, "evict": _evict}[op](s)


# ---------------------------------------------------------------------- work

def work(case):
    e, D, H = (2 if case["dtype"] == "bf16" else 4), case["D"], case["H"]
    if case["op"] == "evict":
        b, f, r, moved, read, kept = case["budget"], case["first"], case["recent"], 0.0, 0, 0
        for n in _lengths(case):
            read, kept = read + n, kept + min(n, b)
            if n > b:
                # rows behind the budget that stay: the last tokens, and their share of the others
                tail = n - b
                safe = min(r, tail, n // 8 if case["born"] else n)
                others = max(1, n - f - r)
                moved += safe + (tail - safe) * max(0.0, min(1.0, (b - f - r) / others))
        stamp = 8 if case["born"] else 4
        return {"bytes": H * (4.0 * D * e * moved + stamp * (read + kept)), "flops": float(H * read)}
    new, length = _counts(case)
    N = sum(new)
    if case["op"] == "keep":
        moved = sum(i != j for k in _kept(case, new) for j, i in enumerate(k))
        return {"bytes": max(1.0, 4.0 * D * e * H * moved + 4 * (moved + 2 * case["B"])), "flops": 0.0}
    if case["op"] == "mass":
        pairs, rows, k = 0, 0, case["block"]
        for n, full in zip(new, length):
            if n:
                past = full - n
                pairs += sum(min(full, ((past + i) // k + 1) * k) for i in range(n)) if k else n * full
                rows += full
        return {"bytes": rows * H * (D * e + 8.0) + N * case["Hq"] * (D * e + 4) + 8 * case["B"],
                "flops": 2.0 * D * pairs * case["Hq"] + 1}
    pairs, size = 0, _sizes(case)
    for t, full in zip(_parents(case, new), length):
        depth = []
        for p in t:
            depth.append(1 + (depth[p] if p >= 0 else 0))
        pairs += sum(depth) + len(t) * (full - len(t))
    rows = sum(full for n, full in zip(new, length) if n)
    pairs = pairs * case["Hq"] + N * case["Hq"] // H * sum(size)
    kv = 2 * D * e * (sum(size) + rows * H) + (4 * sum(size) if case["counts"] else 0)
    return {"bytes": kv + N * case["Hq"] * (2 * D * e + 4) + 4 * N, "flops": 4.0 * D * pairs}


# --------------------------------------------------------------- in 64 bits

def _branch(s, b, full, h, x):
    """The first `full` rows of a branch and head in 64 bits."""
    ids = s["table"][b, : -(-full // s["case"]["page"])].long()
    return x[ids, h].flatten(0, 1)[:full].double()


def exact(case, seed):
    s = prepare(case, seed)
    H, page, op = case["H"], case["page"], case["op"]
    if op == "evict":
        K, V = s["K"].double(), s["V"].double()
        mass, born = s["out_mass"].double(), s["out_born"].double()
        budget, first, recent = case["budget"], case["first"], case["recent"]
        for b, n in enumerate(_lengths(case)):
            ids, q = s["table"][b].long().cpu(), torch.arange(n)
            row = (ids[q // page], q % page)
            for h in range(H):
                drew = s["mass"][row[0].cuda(), h, row[1].cuda()].cpu().double()
                number = s["born"][row[0].cuda(), h, row[1].cuda()].cpu() if case["born"] else q
                last = int(s["total"][b]) if case["born"] else n
                safe = (number < first) | (number >= last - recent)
                key = torch.where(safe, math.inf, drew)
                best = torch.argsort(key, descending=True, stable=True)[:budget].sort().values
                stay, behind = best[best < budget], best[best >= budget]
                free = torch.ones(min(budget, n), dtype=torch.bool)
                free[stay] = False
                to = torch.cat((stay, free.nonzero()[: len(behind), 0]))
                src, dst = [(row[0][x].cuda(), row[1][x].cuda()) for x in (torch.cat((stay, behind)), to)]
                for new, old in ((K, s["K"]), (V, s["V"]), (mass, s["mass"]), (born, s["born"])):
                    new[dst[0], h, dst[1]] = old[src[0], h, src[1]].double()
        return (K, V, mass, None) if case["born"] else (K, V, mass)
    new, length = _counts(case)
    cu = _offsets(new)
    if op == "keep":
        K, V = s["K"].double(), s["V"].double()
        for b, (k, n, full) in enumerate(zip(_kept(case, new), new, length)):
            ids, past = s["table"][b].long(), full - n
            i, j = past + torch.tensor(k, device="cuda", dtype=torch.long), past + torch.arange(len(k), device="cuda")
            for y, x in ((K, s["K"]), (V, s["V"])):
                y[ids[j // page], :, j % page] = x[ids[i // page], :, i % page].double()
        return K, V
    if work(case)["flops"] > 4e12:
        return None
    g = case["Hq"] // H
    if op == "mass":
        mass = s["mass"].double()
        for b, (n, full) in enumerate(zip(new, length)):
            if not n:
                continue
            take = s["take"][cu[b]:cu[b + 1]].long()
            i = torch.arange(full - n, full, device="cuda")
            end = (i // case["block"] + 1) * case["block"] if case["block"] else torch.full_like(i, full)
            hidden = torch.arange(full, device="cuda") >= end[:, None]
            p = torch.arange(full, device="cuda")
            at = s["table"][b].long()[p // page], p % page
            for h in range(H):
                k = _branch(s, b, full, h, s["K"])
                drew = torch.zeros(full, dtype=torch.float64, device="cuda")
                for head in range(h * g, (h + 1) * g):
                    x = s["q"][head, take].double() @ k.T * s["scale"]
                    drew += torch.exp(x - s["lse"][head, take].double()[:, None]).masked_fill(hidden, 0).sum(0)
                old = torch.where(p < full - n, case["decay"] * mass[at[0], h, at[1]], 0)
                mass[at[0], h, at[1]] = old + drew
        return mass, None
    size = _sizes(case)
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    lse = torch.zeros_like(s["lse"], dtype=torch.float64)
    for b, (n, full, tree) in enumerate(zip(new, length, _parents(case, new))):
        if not n:
            continue
        hidden = torch.zeros(n, full, dtype=torch.bool)
        hidden[:, full - n:] = True
        for i in range(n):
            j = i
            while j >= 0:
                hidden[i, full - n + j] = False
                j = tree[j]
        hidden = hidden.cuda()
        for h in range(H):
            k = torch.cat((s["pK"][h, : size[h]].double(), _branch(s, b, full, h, s["K"])))
            v = torch.cat((s["pV"][h, : size[h]].double(), _branch(s, b, full, h, s["V"])))
            x = s["q"][h * g:(h + 1) * g, cu[b]:cu[b + 1]].double() @ k.T * s["scale"]
            if case["counts"]:
                x[..., : size[h]] += s["m"][h, : size[h]].double().log()
            x[..., size[h]:] = x[..., size[h]:].masked_fill(hidden, -torch.inf)
            out[h * g:(h + 1) * g, cu[b]:cu[b + 1]] = torch.softmax(x, -1) @ v
            lse[h * g:(h + 1) * g, cu[b]:cu[b + 1]] = torch.logsumexp(x, -1)
    return out, lse
