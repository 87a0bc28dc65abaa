"""Cases of the paged-cache serving operators: the page plan of a step, rotary positions with the int8 append,
page bounds and page selection, and decode attention over selected pages.

Each case is one call as a serving loop makes it: buffers that such a program keeps (the page pool, block tables,
outputs, workspaces) are made in prepare(), the call's inputs come from the seed.  With `own` false the operators are
computed in their plain form, elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # ---- paged_assign: the page plan of one serving step
        # a small batch that decodes: one token each, now and then a page
        {"name": "assign_decode", "op": "assign", "B": 8, "page": 16, "max_blocks": 512, "ctx": 4096, "chunk": 1, "prefills": 0, "released": 0},
        # a full server: 256 slots of which some start with prompt chunks, some have ended, some find no pages
        {"name": "assign_mixed", "op": "assign", "B": 256, "page": 16, "max_blocks": 2048, "ctx": 24000, "chunk": 8192, "prefills": 31, "released": 17},
        # ---- rope_append: rotate q and k, quantise k and v, store them in their pages
        # decode of 64 sequences (Hq 32, Hkv 8, d 128)
        {"name": "append_decode", "op": "append", "T": 64, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "axes": 1, "adjacent": False, "page": 64, "dtype": "bf16", "skip": 0},
        # an image prompt: time, height and width positions, part of each head rotated, some padded tokens
        {"name": "append_image", "op": "append", "T": 4099, "Hq": 16, "Hkv": 2, "d": 128, "rot": 96, "axes": 3, "adjacent": False, "page": 16, "dtype": "f16", "skip": 5},
        # a long prompt at the widest head dim, adjacent pairs (Hq 16, Hkv 8, d 256)
        {"name": "append_long", "op": "append", "T": 16384, "Hq": 16, "Hkv": 8, "d": 256, "rot": 256, "axes": 1, "adjacent": True, "page": 64, "dtype": "bf16", "skip": 0},
        # ---- page_bounds: the summary that the selection scores, after an append
        {"name": "bounds_decode", "op": "bounds", "B": 64, "Hkv": 8, "d": 128, "page": 64, "ctx": 2048, "new": 1},
        {"name": "bounds_chunk", "op": "bounds", "B": 4, "Hkv": 8, "d": 128, "page": 16, "ctx": 8192, "new": 8192},
        # ---- page_select: score every page of each sequence, keep the best ones
        # one long conversation
        {"name": "select_one", "op": "select", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 64, "ctx": 131072, "keep": 64, "dtype": "bf16"},
        # a decode batch with ragged contexts
        {"name": "select_batch", "op": "select", "B": 64, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 32, "ctx": 32768, "keep": 128, "dtype": "bf16"},
        # ---- sparse decode: attention over each kv head's own page list
        # four sequences, a small budget of small pages
        {"name": "sparse_small", "op": "sparse", "B": 4, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 16, "keep": 32, "ctx": 16384, "dtype": "bf16"},
        # drafts of a speculative step, each with its own list (Hq 4, Hkv 2, d 64)
        {"name": "sparse_drafts", "op": "sparse", "B": 16, "T": 5, "Hq": 4, "Hkv": 2, "d": 64, "page": 32, "keep": 31, "ctx": 8192, "dtype": "f16"},
        # a decode batch of 64 that keeps 4,096 tokens a head
        {"name": "sparse_batch", "op": "sparse", "B": 64, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 64, "keep": 64, "ctx": 16384, "dtype": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["assign", "append", "bounds", "select", "sparse"])
    if op == "assign":
        page = rng.choice([16, 32, 64])
        B = spread(1, 256)
        return {"op": op, "B": B, "page": page, "max_blocks": 32768 // page, "ctx": spread(page, 24000), "chunk": spread(1, 8192),
                "prefills": rng.randrange(0, B // 8 + 1), "released": rng.randrange(0, B // 8 + 1)}
    if op == "append":
        d = rng.choice([32, 64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        T = spread(1, max(8, (16384 * 256 * 8) // (d * Hkv) // 8))
        return {"op": op, "T": T, "Hq": Hkv * rng.choice([1, 2, 4]), "Hkv": Hkv, "d": d, "rot": rng.choice([d, d, d // 2, 3 * d // 4]),
                "axes": rng.choice([1, 1, 2, 3]), "adjacent": rng.random() < 0.5, "page": rng.choice([16, 32, 64]),
                "dtype": rng.choice(["f16", "bf16", "bf16"]), "skip": rng.randrange(0, 4)}
    if op == "bounds":
        return {"op": op, "B": spread(1, 64), "Hkv": rng.choice([1, 2, 4, 8]), "d": rng.choice([32, 64, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
                "ctx": spread(1, 4096), "new": spread(1, 512)}
    if op == "select":
        Hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "B": spread(1, 48), "T": rng.choice([1, 1, 1, 3]), "Hq": Hkv * rng.choice([1, 3, 4, 8, 16]), "Hkv": Hkv, "d": rng.choice([32, 64, 128]),
                "page": rng.choice([16, 32, 64]), "ctx": spread(50, 16384), "keep": spread(4, 200), "dtype": rng.choice(["f16", "bf16", "f32"])}
    Hkv = rng.choice([1, 2, 4, 8])
    return {"op": op, "B": spread(1, 48), "T": rng.choice([1, 1, 1, 3]), "Hq": Hkv * rng.choice([1, 3, 4, 8, 16]), "Hkv": Hkv, "d": rng.choice([32, 64, 128]),
            "page": rng.choice([16, 32, 64]), "keep": spread(4, 24), "ctx": 4096, "dtype": rng.choice(["f16", "bf16"])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(g, lo, hi, shape):  # lo .. hi - 1
    return torch.randint(lo, max(hi, lo + 1), shape, generator=g, device=DEV, dtype=torch.int32)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _pages(n, page):
    return (n + page - 1) // page


def prepare(case, seed):
    s = {"assign": _prepare_assign, "append": _prepare_append, "bounds": _prepare_bounds, "select": _prepare_select,
         "sparse": _prepare_sparse}[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


def _prepare_assign(c, g):
    B, page, nb = c["B"], c["page"], c["max_blocks"]
    cap = nb * page
    ctx = _ints(g, 0, min(c["ctx"], cap - 1) + 1, (B,))
    new = torch.ones(B, dtype=torch.int32, device=DEV)
    order = torch.randperm(B, generator=g, device=DEV)
    started = order[:c["prefills"]]
    new[started] = _ints(g, _pages(c["chunk"], 2), c["chunk"] + 1, (c["prefills"],))
    release = torch.zeros(B, dtype=torch.int32, device=DEV)
    ended = order[c["prefills"]:c["prefills"] + c["released"]]
    release[ended] = 1
    new[ended] = 0
    held = _pages(ctx, page)
    need = int((_pages(ctx + new, page) - held)[release == 0].sum())
    pool = B * _pages(c["ctx"] + 1, page) + _pages(c["prefills"] * c["chunk"], page)
    perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    table = torch.full((B, nb), -1, dtype=torch.int32, device=DEV)
    off = torch.cumsum(held, 0) - held
    at = torch.arange(nb, device=DEV)
    m = at[None] < held[:, None]
    table[m] = perm[(off[:, None] + at)[m]]
    free = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
    rest = perm[int(held.sum()):]
    count = min(rest.numel(), need * 7 // 8 + 1)  # a full server: the last requests may find no page
    free[:count] = rest[:count]
    T = B + c["prefills"] * c["chunk"] + 3  # a step of fixed size: its last tokens are padding
    s = {"ctx": ctx, "new": new, "release": release, "table": table, "free": free, "T": T,
         "count": torch.tensor([count], dtype=torch.int32, device=DEV)}
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    s["out"] = {"seqlens": i32(B), "granted": i32(B), "cu_new": i32(B + 1), "slot_map": i32(T), "token_pos": i32(T), "free_count": i32(1)}
    return s


def _pair_axis(c):
    """Axis of each rotary pair: the first pairs turn with axis 0, then axis 1, and so on."""
    half, axes = c["rot"] // 2, c["axes"]
    return [min(p * axes // half, axes - 1) for p in range(half)]


def _prepare_append(c, g):
    T, Hq, Hkv, d, page, dt = c["T"], c["Hq"], c["Hkv"], c["d"], c["page"], _TYPES[c["dtype"]]
    qkv = _normal(g, T, (Hq + 2 * Hkv) * d).to(dt)  # q, k and v as the fused projection leaves them
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    start = _ints(g, 0, 100000, (c["axes"], 1))
    if T <= 256:  # decode: every token has its own position
        pos = _ints(g, 0, 131072, (c["axes"], T))
    else:
        pos = (start + torch.arange(T, device=DEV, dtype=torch.int32) // torch.tensor([[1], [7], [3]][:c["axes"]], device=DEV)).to(torch.int32)
    inv = (1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])).float()
    num_pages = _pages(T, page) + 1
    slots = torch.arange(T, device=DEV)
    order = torch.randperm(num_pages, generator=g, device=DEV)
    slot_map = (order[slots // page] * page + slots % page).to(torch.int32)
    if c["skip"]:
        slot_map[T - min(c["skip"], T - 1):] = -1
    pool = torch.zeros((2, num_pages, Hkv, page, d), dtype=torch.int8, device=DEV)
    scale = torch.zeros((2, num_pages, Hkv, page), dtype=torch.float32, device=DEV)
    return {"q": q, "k": k, "v": v, "pos": pos if c["axes"] > 1 else pos[0], "inv": inv, "slot_map": slot_map, "pool": pool, "scale": scale, "pages": (pool[0], scale[0], pool[1], scale[1]),
            "axis": bytes(_pair_axis(c)), "q_out": torch.empty((T, Hq, d), dtype=dt, device=DEV), "values": torch.empty(pool.shape, dtype=dt, device=DEV)}


def _block_table(g, held, nb):
    """Each sequence's pages in a shuffled pool that could hold every sequence at full length: (table, pages of the pool)."""
    total = held.numel() * nb
    perm = torch.randperm(total, generator=g, device=DEV, dtype=torch.int32)
    table = torch.zeros((held.numel(), nb), dtype=torch.int32, device=DEV)
    at = torch.arange(nb, device=DEV)
    m = at[None] < held[:, None]
    table[m] = perm[((torch.cumsum(held, 0) - held)[:, None] + at)[m]]
    return table, total


def _prepare_bounds(c, g):
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    lens = _ints(g, 1, c["ctx"] + 1, (B,))
    new = _ints(g, max(1, c["new"] // 2), c["new"] + 1, (B,))
    lens = lens + new
    nb = _pages(c["ctx"] + c["new"], page)
    table, num_pages = _block_table(g, _pages(lens, page).long(), nb)
    k = torch.randint(-127, 128, (num_pages, Hkv, page, d), generator=g, device=DEV, dtype=torch.int8)
    ks = torch.rand((num_pages, Hkv, page), generator=g, device=DEV) * 0.02 + 0.01
    return {"k": k, "ks": ks, "table": table, "lens": lens, "new": new,
            "bounds": torch.zeros((num_pages, Hkv, 2, d), dtype=torch.int8, device=DEV),
            "scale": torch.zeros((num_pages, Hkv), dtype=torch.float32, device=DEV),
            "values": torch.empty((num_pages, Hkv, 2, d), dtype=torch.bfloat16, device=DEV)}


def _prepare_select(c, g):
    B, T, Hq, Hkv, d, page = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page"))
    lens = _ints(g, c["ctx"] // 4, c["ctx"] + 1, (B,)) if B > 1 else torch.full((B,), c["ctx"], dtype=torch.int32, device=DEV)
    nb = _pages(c["ctx"], page)
    table, num_pages = _block_table(g, _pages(lens, page).long(), nb)
    mid = _normal(g, num_pages, Hkv, 1, d) * 20 + _normal(g, 1, Hkv, 1, d) * 20  # channels with a mean of their own
    half = _normal(g, num_pages, Hkv, 2, d).abs() * 10 + 30
    half[:, :, 0].neg_()
    bounds = (mid + half).round_().clamp_(-127, 127).to(torch.int8)
    scale = torch.rand((num_pages, Hkv), generator=g, device=DEV) * 0.01 + 0.02
    q = _normal(g, B, T, Hq, d).to(_TYPES[c["dtype"]])
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"q": q if T > 1 else q[:, 0], "bounds": bounds, "scale": scale, "table": table, "lens": lens,
            "out": {"blocks": i32(B, T, Hkv, c["keep"]), "pages": i32(B, T, Hkv, c["keep"]), "lens": i32(B, T, Hkv)}}


def _prepare_sparse(c, g):
    B, T, Hq, Hkv, d, page, keep = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page", "keep"))
    per = _pages(c["ctx"], page)  # pages that each sequence has in the pool
    num_pages = B * per
    k = torch.randint(-127, 128, (num_pages, Hkv, page, d), generator=g, device=DEV, dtype=torch.int8)
    v = torch.randint(-127, 128, (num_pages, Hkv, page, d), generator=g, device=DEV, dtype=torch.int8)
    ks = torch.rand((num_pages, Hkv, page), generator=g, device=DEV) * 0.02 + 0.01
    vs = torch.rand((num_pages, Hkv, page), generator=g, device=DEV) * 0.02 + 0.01
    chosen = torch.rand((B, T, Hkv, per), generator=g, device=DEV).topk(min(keep, per), -1).indices.sort(-1).values
    pages = torch.zeros((B, T, Hkv, keep), dtype=torch.int32, device=DEV)
    pages[..., :chosen.shape[-1]] = (chosen + torch.arange(B, device=DEV).view(B, 1, 1, 1) * per).to(torch.int32)
    lens = chosen.shape[-1] * page - _ints(g, 0, page, (B, T, Hkv))  # the last page is partly filled
    if B > 2:  # a short conversation and a slot without one
        lens[0] = _ints(g, 1, page * chosen.shape[-1], (T, Hkv))
        lens[1] = 0
    q = _normal(g, B, T, Hq, d).to(_TYPES[c["dtype"]])
    s = {"q": q if T > 1 else q[:, 0], "k": k, "ks": ks, "v": v, "vs": vs, "pages": pages if T > 1 else pages[:, 0], "lens": lens if T > 1 else lens[:, 0]}
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=DEV)
    s["scratch"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)  # one for all layers of a program
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c)


def _lib():
    import w8a8_int8_flashattention_gb300 as sl8
    return sl8


def _own_assign(s, c):
    o = _lib().paged_assign(s["ctx"], s["new"], s["table"], s["free"], s["count"], c["page"], s["T"], release=s["release"], out=s["out"])
    return {**o, "block_table": s["table"], "free_pages": s["free"]}


def _own_append(s, c):
    q = _lib().rope_append(s["q"], s["k"], s["v"], s["pos"], s["inv"], s["slot_map"], *s["pages"], pair_axis=s["axis"],
                           adjacent=c["adjacent"], q_out=s["q_out"])
    return {"q": q, "cache": _values(s["pool"], s["scale"], s["values"]), "scale": s["scale"]}


def _own_bounds(s, c):
    _lib().page_bounds(s["k"], s["ks"], s["table"], s["lens"], s["bounds"], s["scale"], new_lens=s["new"], max_new=c["new"])
    return {"bounds": _values(s["bounds"], s["scale"][:, :, None], s["values"]), "scale": s["scale"]}


def _own_select(s, c):
    return _lib().page_select(s["q"], s["bounds"], s["scale"], s["table"], s["lens"], c["page"], c["keep"], first=1, last=2, out=s["out"])


def _own_sparse(s, c):
    out, lse = _lib().attn_int8_sparse_decode(s["q"], s["k"], s["ks"], s["v"], s["vs"], s["pages"], s["lens"], workspace=s["scratch"],
                                              out=s["out"], lse=s["lse"], return_lse=True)
    return {"out": out, "lse": lse}


_own = {"assign": _own_assign, "append": _own_append, "bounds": _own_bounds, "select": _own_select, "sparse": _own_sparse}


def _values(codes, scale, into):
    """What 8-bit codes stand for."""
    return torch.mul(codes, scale.unsqueeze(-1), out=into)


def _div(x, y):
    """x / y in the IEEE rounding of 32 bits, elementwise (a division by a number becomes a product)."""
    return x / torch.as_tensor(y, dtype=torch.float32, device=x.device).expand_as(x)


def _codes(x, scale):
    """Codes of rows with one scale each; all zero where the scale is zero."""
    return torch.where(scale == 0, torch.zeros_like(x), torch.round(_div(x, scale)).clamp(-127, 127))


def _plain_assign(s, c):
    page, T, table, free = c["page"], s["T"], s["table"], s["free"]
    B, nb = table.shape
    at = torch.arange(nb, device=DEV)
    gone = s["release"] != 0
    ctx = s["ctx"].long()
    back = torch.where(gone, _pages(ctx, page), 0)
    m = at[None] < back[:, None]
    free[(s["count"].long() + torch.cumsum(back, 0)[:, None] - back[:, None] + at)[m]] = table[m]
    have = s["count"].long() + back.sum()
    ctx, new = torch.where(gone, 0, ctx), s["new"].long()
    cu = torch.cumsum(new, 0)
    ok = (ctx + new <= nb * page) & (cu <= T)
    need = torch.where(ok, _pages(ctx + new, page) - _pages(ctx, page), 0)
    upto = torch.cumsum(need, 0)
    ok &= (need == 0) | (upto <= have)
    taken = torch.where(ok, need, 0)
    j = at[None] - _pages(ctx, page)[:, None]
    m = (j >= 0) & (j < taken[:, None])
    table[m] = free[(have - 1 - (upto[:, None] - need[:, None] + j))[m]]
    granted = torch.where(ok, new, 0)
    i = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu, i, right=True).clamp(max=B - 1)
    inside = i < cu[-1]
    pos = torch.where(inside, ctx[b] + i - (cu - new)[b], 0)
    slot = table[b, (pos // page).clamp(max=nb - 1)].long() * page + pos % page
    i32 = torch.int32
    return {"seqlens": (ctx + granted).to(i32), "granted": granted.to(i32), "cu_new": torch.cat([cu[:1] * 0, cu]).to(i32),
            "slot_map": torch.where(inside & ok[b], slot, -1).to(i32), "token_pos": pos.to(i32), "free_count": (have - taken.sum()).to(i32).view(1),
            "block_table": table, "free_pages": free}


def _turn(x, cos, sin, rot, adjacent):
    """The first rot channels of each row turned by its angles."""
    y = x.float()
    if adjacent:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, y[..., rot:]), -1)


def _plain_append(s, c):
    rot, pool, scale, page = c["rot"], s["pool"], s["scale"], c["page"]
    axis = torch.tensor(list(s["axis"]), device=DEV)
    pos = s["pos"].view(c["axes"], -1)
    angle = pos[axis].T.double() * s["inv"].double()  # far positions: 32 bits would lose the angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _turn(s["q"], cos, sin, rot, c["adjacent"]).to(s["q"].dtype)
    t = (s["slot_map"] >= 0).nonzero()[:, 0]
    slot = s["slot_map"][t].long()
    for i, x in enumerate((_turn(s["k"], cos, sin, rot, c["adjacent"]), s["v"].float())):
        x = x[t]
        sc = _div(x.abs().amax(-1), 127.0)
        pool[i][slot // page, :, slot % page] = _codes(x, sc[..., None]).to(torch.int8)
        scale[i][slot // page, :, slot % page] = sc
    return {"q": q, "cache": _values(pool, scale, s["values"]), "scale": scale}


def _plain_bounds(s, c):
    page, lens, new = c["page"], s["lens"], s["new"]
    first, last = (lens - new) // page, (lens - 1) // page
    at = torch.arange(s["table"].shape[1], device=DEV)
    m = (at >= first[:, None]) & (at <= last[:, None])
    p = s["table"][m].long()  # the pages that took tokens, and how many each holds
    held = (lens[:, None] - at * page).clamp(max=page)[m]
    there = (torch.arange(page, device=DEV) < held[:, None])[:, None]
    ks = torch.where(there, s["ks"][p], 0.0)
    sc = ks.amax(-1)
    part = _div(ks, torch.where(sc == 0, 1.0, sc)[..., None])
    x = s["k"][p].float() * part[..., None]  # keys in steps of the page's largest row scale
    lo = torch.where(there[..., None], x, math.inf).amin(2)
    hi = torch.where(there[..., None], x, -math.inf).amax(2)
    s["bounds"][p] = torch.stack((torch.floor(lo), torch.ceil(hi)), 2).to(torch.int8)
    s["scale"][p] = sc
    return {"bounds": _values(s["bounds"], s["scale"][:, :, None], s["values"]), "scale": s["scale"]}


def _quantised(q):
    x = q.float()
    sc = _div(x.abs().amax(-1), 127.0)
    return _codes(x, sc[..., None]), sc


def _plain_select(s, c):
    B, T, Hq, Hkv, d, page, keep = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page", "keep"))
    table, nb = s["table"], s["table"].shape[1]
    codes, sc = _quantised(s["q"].view(B, T, Hkv, Hq // Hkv, d))
    box = s["bounds"][table.long()].float()  # [B, blocks, Hkv, 2, d]
    dots = torch.einsum("btkgd,bnkd->btkgn", codes.clamp(max=0), box[..., 0, :]) + torch.einsum("btkgd,bnkd->btkgn", codes.clamp(min=0), box[..., 1, :])
    score = (dots * s["scale"][table.long()].permute(0, 2, 1)[:, None, :, None] * sc[..., None]).amax(3)
    lens = (s["lens"][:, None] - T + 1 + torch.arange(T, device=DEV)).clamp(min=0)  # of each query's row
    n = _pages(lens, page)[..., None, None]
    at = torch.arange(nb, device=DEV)
    score = torch.where((at < 1) | (at >= n - 2), math.inf, score)  # the first page and the last two are always kept
    score = torch.where(at < n, score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    if best.shape[-1] < keep:
        best = torch.cat((best, best.new_full((*best.shape[:-1], keep - best.shape[-1]), nb)), -1)
    best = torch.where(best < n, best, nb).sort(-1).values
    there = best < n
    blocks = torch.where(there, best, -1)
    pages = torch.where(there, table[:, None, None].expand(B, T, Hkv, nb).gather(-1, best.clamp(max=nb - 1)), -1)
    kept = there.sum(-1)
    tokens = torch.where(kept > 0, kept * page - (n[..., 0] * page - lens[..., None]), 0)
    return {"blocks": blocks.to(torch.int32), "pages": pages.to(torch.int32), "lens": tokens.to(torch.int32)}


def _plain_sparse(s, c):
    B, T, Hq, Hkv, d, page, keep = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page", "keep"))
    codes, sc = _quantised(s["q"].view(B, T, Hkv, Hq // Hkv, d))
    p, h = s["pages"].view(B, T, Hkv, keep).long(), torch.arange(Hkv, device=DEV)[:, None]
    lens = s["lens"].view(B, T, Hkv)
    k, ks = s["k"][p, h].float().flatten(3, 4), s["ks"][p, h].flatten(3)
    x = torch.einsum("btkgd,btknd->btkgn", codes, k) * (ks[..., None, :] * (sc / math.sqrt(d))[..., None])
    x = torch.where(torch.arange(keep * page, device=DEV) < lens[..., None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    v = s["v"][p, h].float().flatten(3, 4) * s["vs"][p, h].flatten(3)[..., None]
    o = torch.einsum("btkgn,btknd->btkgd", e / torch.where(total == 0, 1.0, total), v)
    return {"out": o.to(s["q"].dtype).view(s["q"].shape), "lse": (m + torch.log(total)).view(s["lse"].shape)}


_plain = {"assign": _plain_assign, "append": _plain_append, "bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse}


# ---------------------------------------------------------------- what a pass cannot do without

def work(c):
    """Bytes read once and written once, and the operations of the products; counts of ragged cases are their means."""
    size = {"f16": 2, "bf16": 2, "f32": 4}.get(c.get("dtype"), 4)
    if c["op"] == "assign":
        step = c["B"] + c["prefills"] * c["chunk"]
        moved = c["prefills"] * c["chunk"] * 3 // 4 // c["page"] + c["released"] * c["ctx"] // 2 // c["page"]
        return {"bytes": 4 * (6 * c["B"] + 2 * step + 2 * moved), "flops": 0}
    if c["op"] == "append":
        T, d = c["T"], c["d"]
        rows = _pages(T, c["page"]) * c["page"] + c["page"]  # the pool's rows, returned as values
        return {"bytes": T * d * size * (2 * c["Hq"] + 2 * c["Hkv"]) + 2 * T * c["Hkv"] * (d + 4) + 4 * T * (1 + c["axes"])
                + 2 * rows * c["Hkv"] * d * size, "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "bounds":
        mean, page = (3 * c["new"] + 3) // 4, c["page"]
        touched = c["B"] * ((mean + page - 2) // page + 1)
        pool = c["B"] * _pages(c["ctx"] + c["new"], page)  # the summary is returned whole, as values
        rows = touched * page if c["new"] > page else touched * (page // 2)
        return {"bytes": rows * c["Hkv"] * (c["d"] + 4) + touched * c["Hkv"] * (2 * c["d"] + 4) + pool * c["Hkv"] * (2 * c["d"] * 2), "flops": 0}
    d, T, group = c["d"], c["T"], c["Hq"] // c["Hkv"]
    if c["op"] == "select":
        mean = c["ctx"] if c["B"] == 1 else c["ctx"] * 5 // 8
        pages = c["B"] * _pages(mean, c["page"])
        return {"bytes": pages * (c["Hkv"] * (2 * d + 4) + 4) + c["B"] * T * (c["Hq"] * d * size + c["Hkv"] * 4 * (2 * c["keep"] + 1)),
                "flops": 4 * pages * T * c["Hq"] * d}
    tokens = c["B"] * T * c["Hkv"] * min(c["keep"], _pages(c["ctx"], c["page"])) * c["page"] * (1 if c["B"] <= 2 else (c["B"] - 1.5) / c["B"])
    return {"bytes": tokens * (2 * d + 8) + 2 * c["B"] * T * c["Hq"] * d * size, "flops": 4 * tokens * group * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s, case)
    if case["op"] == "bounds":
        return _exact_bounds(s, case)
    if case["op"] == "sparse":
        return _exact_sparse(s, case)
    return None  # page plans and selections are whole numbers


def _exact_append(s, c):
    """Rotation as a product of complex numbers; the stored rows are the nearest multiples of their scales."""
    rot, half, page = c["rot"], c["rot"] // 2, c["page"]
    pos = s["pos"].view(c["axes"], -1).double()
    turns = torch.stack([pos[a] for a in s["axis"]], 1) * s["inv"].double()
    unit = torch.polar(torch.ones_like(turns), turns)[:, None]

    def rotated(x):
        y = x.double().clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if c["adjacent"] else (slice(0, half), slice(half, rot))
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    cache = torch.zeros(s["pool"].shape, dtype=torch.float64, device=DEV)
    scale = torch.zeros(s["scale"].shape, dtype=torch.float64, device=DEV)
    at = torch.nonzero(s["slot_map"] >= 0)[:, 0]
    page_of, row = s["slot_map"][at].long() // page, s["slot_map"][at].long() % page
    for i, x in enumerate((rotated(s["k"]), s["v"].double())):
        step = x[at].abs().amax(-1) / 127
        cache[i][page_of, :, row] = torch.round(x[at] / step[..., None]) * step[..., None]
        scale[i][page_of, :, row] = step
    return {"q": rotated(s["q"]), "cache": cache, "scale": scale}


def _exact_bounds(s, c):
    """The least and the largest key of each channel in steps of the page's largest row scale, rounded outwards."""
    page = c["page"]
    out = torch.zeros(s["bounds"].shape, dtype=torch.float64, device=DEV)
    scale = torch.zeros(s["scale"].shape, dtype=torch.float64, device=DEV)
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        first = (n - m) // page
        p = s["table"][b, first:_pages(n, page)].long()
        fill = p.numel() * page - (n - first * page)
        rows = s["ks"][p].double().transpose(1, 2).flatten(0, 1)  # [rows, Hkv]
        rows[rows.shape[0] - fill:] = 0
        step = rows.unflatten(0, (p.numel(), page)).amax(1)
        x = s["k"][p].double().transpose(1, 2).flatten(0, 1) * (rows / step.repeat_interleave(page, 0))[..., None]
        x[x.shape[0] - fill:] = math.nan
        x = x.unflatten(0, (p.numel(), page))
        lo, hi = torch.nan_to_num(x, nan=math.inf).amin(1), torch.nan_to_num(x, nan=-math.inf).amax(1)
        out[p] = torch.stack((lo.floor(), hi.ceil()), 2) * step[..., None, None]
        scale[p] = step
    return {"bounds": out, "scale": scale}


def _exact_sparse(s, c):
    B, T, Hq, Hkv, d, page, keep = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page", "keep"))
    q = s["q"].view(B, T, Hkv, Hq // Hkv, d).float()
    step = q.abs().amax(-1, keepdim=True) / torch.full((1,), 127.0, device=DEV)  # the query's codes are part of the definition
    q = torch.where(step > 0, torch.round(q / step).clamp(-127, 127), 0.0).double() * step.double()
    pages, lens = s["pages"].view(B, T, Hkv, keep), s["lens"].view(B, T, Hkv).tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        for t in range(T):
            for h in range(Hkv):
                n = lens[b][t][h]
                if n == 0:
                    continue
                p = pages[b, t, h, :_pages(n, page)].long()
                k = (s["k"][p, h].double() * s["ks"][p, h].double()[..., None]).flatten(0, 1)[:n]
                v = (s["v"][p, h].double() * s["vs"][p, h].double()[..., None]).flatten(0, 1)[:n]
                x = q[b, t, h] @ k.T / math.sqrt(d)
                lse[b, t, h] = torch.logsumexp(x, -1)
                out[b, t, h] = torch.softmax(x, -1) @ v
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["lse"].shape)}
