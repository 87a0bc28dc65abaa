"""Cases of the paged 4-bit KV cache: rotary positions with the 4-bit append, reading a cache back as dense keys and
values, and decode attention over the 4-bit pages.

Each case is one call as a serving loop makes it: buffers that such a program keeps (the page pool, block tables,
outputs, workspaces) are made in prepare(), the call's inputs come from the seed.  With `own` false the operators are
computed in their plain form, elementary torch operations.

The cache: a row of d channels (one token, one kv head) is cut into groups of 32 consecutive channels.  Each group has a
bf16 scale s = bf16(max|x| / 7) and codes round-half-even(x / s), clamped to +-7, held as code + 8 in 4 bits: byte i of a
row holds channel 2 i in its low half and channel 2 i + 1 in its high half.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32  # channels that share a scale


def listed():
    return [
        # ---- append: rotate q and k, quantise k and v to 4 bits, store them in their pages
        # decode of 64 sequences (Hq 32, Hkv 8, d 128)
        {"name": "append4_decode", "op": "append", "T": 64, "Hq": 32, "Hkv": 8, "d": 128, "rot": 128, "axes": 1, "adjacent": False, "page": 64, "dtype": "bf16", "skip": 0, "mean": False},
        # an image prompt: time, height and width positions, part of each head rotated, the plain channels with an
        # offset of their own that is taken off before quantising, some padded tokens
        {"name": "append4_image", "op": "append", "T": 4099, "Hq": 16, "Hkv": 2, "d": 128, "rot": 96, "axes": 3, "adjacent": False, "page": 16, "dtype": "f16", "skip": 5, "mean": True},
        # a long prompt at the widest head dim, adjacent pairs (Hq 16, Hkv 8, d 256)
        {"name": "append4_long", "op": "append", "T": 16384, "Hq": 16, "Hkv": 8, "d": 256, "rot": 256, "axes": 1, "adjacent": True, "page": 64, "dtype": "bf16", "skip": 0, "mean": False},
        # ---- read: the cache of a prompt's prefix as dense keys and values, for the prefill of its next chunk
        # one short prefix of a small model (Hkv 2, d 64)
        {"name": "read4_prefix", "op": "read", "B": 1, "Hkv": 2, "d": 64, "page": 16, "ctx": 1000, "packed": False, "dtype": "f16", "mean": False},
        # ragged prefixes into a packed batch that has room for each one's next chunk (Hkv 8, d 128)
        {"name": "read4_packed", "op": "read", "B": 8, "Hkv": 8, "d": 128, "page": 64, "ctx": 8192, "packed": True, "dtype": "bf16", "mean": True},
        # one long conversation (Hkv 8, d 128)
        {"name": "read4_long", "op": "read", "B": 1, "Hkv": 8, "d": 128, "page": 64, "ctx": 131072, "packed": False, "dtype": "bf16", "mean": False},
        # ---- attend: decode attention over the pages
        # four sequences of moderate length (Hq 32, Hkv 8, d 128)
        {"name": "attend4_small", "op": "attend", "B": 4, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 16, "ctx": 2048, "tree": False, "dtype": "bf16"},
        # one long conversation
        {"name": "attend4_one", "op": "attend", "B": 1, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 64, "ctx": 131072, "tree": False, "dtype": "bf16"},
        # a tree of drafts in a speculative step
        {"name": "attend4_drafts", "op": "attend", "B": 16, "T": 5, "Hq": 32, "Hkv": 8, "d": 128, "page": 32, "ctx": 8192, "tree": True, "dtype": "bf16"},
        # many query heads on few kv heads of a small head dim (Hq 32, Hkv 2, d 64)
        {"name": "attend4_d64", "op": "attend", "B": 48, "T": 1, "Hq": 32, "Hkv": 2, "d": 64, "page": 16, "ctx": 16384, "tree": False, "dtype": "f16"},
        # a decode batch of 64 with ragged contexts (Hq 32, Hkv 8, d 128)
        {"name": "attend4_batch", "op": "attend", "B": 64, "T": 1, "Hq": 32, "Hkv": 8, "d": 128, "page": 64, "ctx": 8192, "tree": False, "dtype": "bf16"},
        # the widest head dim, queries and outputs in 32 bits (Hq 16, Hkv 8, d 256)
        {"name": "attend4_d256", "op": "attend", "B": 32, "T": 1, "Hq": 16, "Hkv": 8, "d": 256, "page": 32, "ctx": 4096, "tree": False, "dtype": "f32"},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["append", "read", "attend", "attend"])
    if op == "append":
        d = rng.choice([32, 64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        T = spread(1, max(8, (16384 * 256 * 8) // (d * Hkv) // 8))
        return {"op": op, "T": T, "Hq": Hkv * rng.choice([1, 2, 4]), "Hkv": Hkv, "d": d, "rot": rng.choice([d, d, d // 2, 3 * d // 4]),
                "axes": rng.choice([1, 1, 2, 3]), "adjacent": rng.random() < 0.5, "page": rng.choice([16, 32, 64]),
                "dtype": rng.choice(["f16", "bf16", "bf16"]), "skip": rng.randrange(0, 4), "mean": rng.random() < 0.5}
    if op == "read":
        return {"op": op, "B": spread(1, 8), "Hkv": rng.choice([1, 2, 4, 8]), "d": rng.choice([32, 64, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
                "ctx": spread(1, 8000), "packed": rng.random() < 0.5, "dtype": rng.choice(["f16", "bf16", "f32"]), "mean": rng.random() < 0.5}
    Hkv = rng.choice([1, 2, 4, 8])
    T, Hq, d, ctx = rng.choice([1, 1, 1, 2, 4, 7]), Hkv * rng.choice([1, 3, 4, 8, 16]), rng.choice([32, 64, 128, 256]), spread(16, 6000)
    most = int(2.5e10 / (2.25 * ctx * T * Hq * d))  # sequences that cost as much as the largest listed case
    return {"op": op, "B": spread(1, max(1, min(48, most))), "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "page": rng.choice([16, 32, 64]), "ctx": ctx,
            "tree": T > 1 and rng.random() < 0.5, "dtype": rng.choice(["f16", "bf16", "f32"])}


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
    s = {"append": _prepare_append, "read": _prepare_read, "attend": _prepare_attend}[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


def _pair_axis(c):
    """Axis of each rotary pair: the first pairs turn with axis 0, then axis 1, and so on."""
    half, axes = c["rot"] // 2, c["axes"]
    return [min(p * axes // half, axes - 1) for p in range(half)]


def _prepare_append(c, g):
    T, Hq, Hkv, d, page, dt = c["T"], c["Hq"], c["Hkv"], c["d"], c["page"], _TYPES[c["dtype"]]
    x = _normal(g, T, Hq + 2 * Hkv, d).clamp_(-1.9, 1.9)  # rows that a norm has bounded
    mean = None
    if c["mean"]:  # what a calibration found: the channels that do not turn have offsets
        mean = _normal(g, Hkv, d)
        mean[:, :c["rot"]] = 0
        x[:, Hq:Hq + Hkv] += mean
    qkv = x.to(dt).flatten(1)  # q, k and v as the fused projection leaves them
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
    pool, scale = _empty_pool(num_pages, Hkv, page, d)
    return {"q": q, "k": k, "v": v, "pos": pos if c["axes"] > 1 else pos[0], "inv": inv, "slot_map": slot_map, "mean": mean,
            "pool": pool, "scale": scale, "pages": (pool[0], scale[0], pool[1], scale[1]), "axis": bytes(_pair_axis(c)),
            "q_out": torch.empty((T, Hq, d), dtype=dt, device=DEV), "values": torch.empty((2, num_pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV),
            "every": torch.arange(num_pages, device=DEV, dtype=torch.int32).view(-1, 1), "full": torch.full((num_pages,), page, dtype=torch.int32, device=DEV)}


def _empty_pool(num_pages, Hkv, page, d):
    """Codes and scales of keys and values, all zero."""
    return (torch.full((2, num_pages, Hkv, page, d // 2), 0x88, dtype=torch.uint8, device=DEV),
            torch.zeros((2, num_pages, Hkv, page, d // GROUP), dtype=torch.bfloat16, device=DEV))


def _filled_pool(g, num_pages, Hkv, page, d):
    """A pool as an append of bell-shaped rows leaves it."""
    codes = torch.empty((2, num_pages, Hkv, page, d // 2), dtype=torch.uint8, device=DEV)
    for i in range(2):
        x = _normal(g, num_pages, Hkv, page, d).mul_(3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        torch.bitwise_or(x[..., 0::2], x[..., 1::2] << 4, out=codes[i])
    scale = (torch.rand((2, num_pages, Hkv, page, d // GROUP), generator=g, device=DEV) * 0.2 + 0.2).to(torch.bfloat16)
    return codes, scale


def _block_table(g, held, nb):
    """Each sequence's pages in a shuffled pool that could hold every sequence at full length: (table, pages of the pool)."""
    total = held.numel() * nb
    perm = torch.randperm(total, generator=g, device=DEV, dtype=torch.int32)
    table = torch.zeros((held.numel(), nb), dtype=torch.int32, device=DEV)
    at = torch.arange(nb, device=DEV)
    m = at[None] < held[:, None]
    table[m] = perm[((torch.cumsum(held, 0) - held)[:, None] + at)[m]]
    return table, total


def _lengths(c, g):
    """Ragged contexts up to c["ctx"]; a single sequence has all of it."""
    if c["B"] == 1:
        return torch.full((1,), c["ctx"], dtype=torch.int32, device=DEV)
    return _ints(g, max(1, c["ctx"] // 8), c["ctx"] + 1, (c["B"],))


def _prepare_read(c, g):
    B, Hkv, d, page, ctx = c["B"], c["Hkv"], c["d"], c["page"], c["ctx"]
    lens = _lengths(c, g)
    table, num_pages = _block_table(g, _pages(lens, page).long(), _pages(ctx, page))
    pool, scale = _filled_pool(g, num_pages, Hkv, page, d)
    mean = _normal(g, Hkv, d) if c["mean"] else None
    cu = None
    if c["packed"]:  # room for 64 more tokens behind each prefix
        cu = torch.arange(B + 1, device=DEV, dtype=torch.int32) * (ctx + 64)
    shape = (B * (ctx + 64), Hkv, d) if c["packed"] else (B, Hkv, ctx, d)
    out = torch.zeros((2, *shape), dtype=_TYPES[c["dtype"]], device=DEV)
    return {"pool": pool, "scale": scale, "pages": (pool[0], scale[0], pool[1], scale[1]), "table": table, "lens": lens, "cu": cu, "mean": mean, "out": out}


def _prepare_attend(c, g):
    B, T, Hq, Hkv, d, page = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page"))
    lens = _lengths(c, g)
    if B > 8:  # a short conversation and a slot without one
        lens[0] = _ints(g, 1, 2 * T + 2, (1,))
        lens[1] = 0
    table, num_pages = _block_table(g, _pages(lens, page).long(), _pages(c["ctx"], page))
    pool, scale = _filled_pool(g, num_pages, Hkv, page, d)
    q = _normal(g, B, T, Hq, d).to(_TYPES[c["dtype"]])
    mask = None
    if c["tree"]:  # each draft sees itself and the drafts that led to it
        parent = [_ints(g, 0, t, (B,)).long() for t in range(1, T)]
        mask = torch.zeros((B, T), dtype=torch.int32, device=DEV)
        mask[:, 0] = 1
        for t in range(1, T):
            mask[:, t] = mask.gather(1, parent[t - 1][:, None])[:, 0] | (1 << t)
    s = {"q": q if T > 1 else q[:, 0], "pool": pool, "scale": scale, "pages": (pool[0], scale[0], pool[1], scale[1]), "table": table, "lens": lens, "mask": mask}
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


def _own_append(s, c):
    sl8, v = _lib(), s["values"]
    q = sl8.rope_append_int4(s["q"], s["k"], s["v"], s["pos"], s["inv"], s["slot_map"], *s["pages"], pair_axis=s["axis"],
                             adjacent=c["adjacent"], q_out=s["q_out"], k_mean=s["mean"])
    # what the whole pool stands for: every page as a sequence of its own
    sl8.paged_read_int4(*s["pages"], s["every"], s["full"], max_seqlen=c["page"], k_mean=s["mean"], k_out=v[0], v_out=v[1])
    return {"q": q, "k": v[0], "v": v[1]}


def _own_read(s, c):
    k, v = _lib().paged_read_int4(*s["pages"], s["table"], s["lens"], cu_seqlens=s["cu"], max_seqlen=c["ctx"], k_mean=s["mean"],
                                  k_out=s["out"][0], v_out=s["out"][1])
    return {"k": k, "v": v}


def _own_attend(s, c):
    out, lse = _lib().attn_int4_paged_decode(s["q"], *s["pages"], s["table"], s["lens"], tree_mask=s["mask"], workspace=s["scratch"],
                                             out=s["out"], lse=s["lse"], return_lse=True)
    return {"out": out, "lse": lse}


_own = {"append": _own_append, "read": _own_read, "attend": _own_attend}


def _div(x, y):
    """x / y in the IEEE rounding of 32 bits, elementwise (a division by a number becomes a product)."""
    return x / torch.as_tensor(y, dtype=torch.float32, device=x.device).expand_as(x)


def _quantised(x):
    """Packed codes and bf16 scales of fp32 rows."""
    x = x.unflatten(-1, (-1, GROUP))
    sc = _div(x.abs().amax(-1), 7.0).to(torch.bfloat16)
    s = sc.float()[..., None]
    codes = torch.where(s == 0, 0.0, torch.round(_div(x, s)).clamp(-7, 7)).flatten(-2).add(8).to(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), sc


def _values(codes, scale):
    """What packed codes and their scales stand for, fp32."""
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (x.unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


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
    k = _turn(s["k"], cos, sin, rot, c["adjacent"])
    if s["mean"] is not None:
        k = k - s["mean"]
    t = (s["slot_map"] >= 0).nonzero()[:, 0]
    slot = s["slot_map"][t].long()
    (pool[0][slot // page, :, slot % page], scale[0][slot // page, :, slot % page]) = _quantised(k[t])
    (pool[1][slot // page, :, slot % page], scale[1][slot // page, :, slot % page]) = _quantised(s["v"][t].float())
    k = _values(pool[0], scale[0])
    if s["mean"] is not None:
        k = k + s["mean"][:, None]
    return {"q": q, "k": k.to(torch.bfloat16), "v": _values(pool[1], scale[1]).to(torch.bfloat16)}


def _plain_read(s, c):
    page, lens, out = c["page"], s["lens"], s["out"]
    p = s["table"].long()
    i = torch.arange(c["ctx"], device=DEV)
    there = i < lens[:, None]
    for n, mean in ((0, s["mean"]), (1, None)):
        x = _values(s["pool"][n][p], s["scale"][n][p])  # [B, blocks, Hkv, page, d]
        x = x.transpose(1, 2).flatten(2, 3)[:, :, :c["ctx"]]
        if mean is not None:
            x = x + mean[:, None]
        if c["packed"]:
            row = (s["cu"][:-1, None] + i)[there].long()
            out[n][row] = x.transpose(1, 2)[there].to(out.dtype)
        else:
            torch.where(there[:, None, :, None], x.to(out.dtype), out[n], out=out[n])
    return {"k": out[0], "v": out[1]}


def _plain_attend(s, c):
    B, T, Hq, Hkv, d, page = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page"))
    q = s["q"].view(B, T, Hkv, Hq // Hkv, d).float()
    step = _div(q.abs().amax(-1), 127.0)[..., None]  # the query rows are quantised to int8, as in every decode here
    codes = torch.where(step == 0, 0.0, torch.round(_div(q, torch.where(step == 0, 1.0, step))).clamp(-127, 127))
    p = s["table"].long()
    k = _values(s["pool"][0][p], s["scale"][0][p]).transpose(1, 2).flatten(2, 3)  # [B, Hkv, tokens, d]
    x = torch.einsum("btkgd,bknd->btkgn", codes, k) * (step / math.sqrt(d))
    del k
    at, first = torch.arange(x.shape[-1], device=DEV), (s["lens"] - T).view(B, 1, 1)  # of the drafts
    u = at - first
    if s["mask"] is None:
        seen = u <= torch.arange(T, device=DEV).view(1, T, 1)
    else:
        seen = (u < 0) | ((s["mask"][..., None] >> u.clamp(0, 31)) & 1).bool()
    seen = (seen & (at < s["lens"].view(B, 1, 1)))[:, :, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    v = _values(s["pool"][1][p], s["scale"][1][p]).transpose(1, 2).flatten(2, 3)
    o = torch.einsum("btkgn,bknd->btkgd", e / torch.where(total == 0, 1.0, total), v)
    return {"out": o.to(s["q"].dtype).reshape(s["q"].shape), "lse": (m + torch.log(total)).reshape(s["lse"].shape)}


_plain = {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}


# ---------------------------------------------------------------- what a pass cannot do without

def work(c):
    """Bytes read once and written once, and the operations of the products; counts of ragged cases are their means."""
    size = {"f16": 2, "bf16": 2, "f32": 4}[c["dtype"]]
    d, Hkv, page = c["d"], c["Hkv"], c["page"]
    row = d // 2 + d // GROUP * 2  # bytes of a cached row: codes and scales
    if c["op"] == "append":
        T = c["T"]
        rows = _pages(T, page) * page + page  # the pool's rows, returned as values
        return {"bytes": T * d * size * (2 * c["Hq"] + 2 * Hkv) + 2 * T * Hkv * row + 4 * T * (1 + c["axes"]) + 2 * rows * Hkv * (row + 2 * d),
                "flops": 3 * T * (c["Hq"] + Hkv) * c["rot"]}
    mean = c["ctx"] if c["B"] == 1 else max(1, c["ctx"] * 9 // 16)
    if c["op"] == "read":
        return {"bytes": 2 * c["B"] * mean * Hkv * (row + d * size), "flops": 0}
    tokens = (c["B"] if c["B"] <= 8 else c["B"] - 2) * mean
    return {"bytes": 2 * tokens * Hkv * row + 2 * c["B"] * c["T"] * c["Hq"] * d * size, "flops": 4 * tokens * c["T"] * c["Hq"] * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s, case)


def _meant(codes, scale):
    """Rows of 64-bit values from packed rows [n, d / 2] and scales [n, d / 32]."""
    x = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=DEV)
    x[:, 0::2] = (codes % 16).double()
    x[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    return (x - 8) * scale.double().repeat_interleave(GROUP, 1)


def _exact_append(s, c):
    """Rotation as a product of complex numbers; a stored value is the nearest multiple of its group's scale."""
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

    found = {"q": rotated(s["q"])}
    mean = torch.zeros((c["Hkv"], c["d"]), dtype=torch.float64, device=DEV) if s["mean"] is None else s["mean"].double()
    at = torch.nonzero(s["slot_map"] >= 0)[:, 0]
    page_of, row = s["slot_map"][at].long() // page, s["slot_map"][at].long() % page
    for name, x, off in (("k", rotated(s["k"]) - mean, mean), ("v", s["v"].double(), torch.zeros_like(mean))):
        kept = off[:, None].expand(c["Hkv"], page, c["d"]).repeat(s["pool"].shape[1], 1, 1, 1)
        step = (x[at].unflatten(-1, (-1, GROUP)).abs().amax(-1) / 7).float().to(torch.bfloat16).double().repeat_interleave(GROUP, -1)
        near = torch.where(step > 0, torch.round(x[at] / step) * step, 0.0)
        kept[page_of, :, row] = torch.minimum(torch.maximum(near, -7 * step), 7 * step) + off
        found[name] = kept
    return found


def _exact_read(s, c):
    page, out = c["page"], torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        p = s["table"][b, :_pages(n, page)].long()
        for i in range(2):
            x = s["pool"][i][p].transpose(0, 1).flatten(1, 2)[:, :n]  # [Hkv, n, d / 2]
            y = torch.stack([_meant(x[h], s["scale"][i][p, h].flatten(0, 1)[:n]) for h in range(c["Hkv"])])
            if i == 0 and s["mean"] is not None:
                y = y + s["mean"].double()[:, None]
            if c["packed"]:
                first = int(s["cu"][b])
                out[i, first:first + n] = y.transpose(0, 1)
            else:
                out[i, b, :, :n] = y
    return {"k": out[0], "v": out[1]}


def _exact_attend(s, c):
    B, T, Hq, Hkv, d, page = (c[x] for x in ("B", "T", "Hq", "Hkv", "d", "page"))
    q = s["q"].view(B, T, Hkv, Hq // Hkv, d).float()
    step = q.abs().amax(-1, keepdim=True) / torch.full((1,), 127.0, device=DEV)  # the query's codes are part of the definition
    q = torch.where(step > 0, torch.round(q / step).clamp(-127, 127), 0.0).double() * step.double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    lens, mask = s["lens"].tolist(), None if s["mask"] is None else s["mask"].tolist()
    for b in range(B):
        n = lens[b]
        p = s["table"][b, :_pages(n, page)].long()
        rows = []  # tokens that each query sees
        for t in range(T):
            drafts = [n - T + u for u in range(T) if (u <= t if mask is None else mask[b][t] >> u & 1)]
            keep = torch.zeros(n, dtype=torch.bool, device=DEV)
            keep[:max(0, n - T)] = True
            keep[[i for i in drafts if i >= 0]] = True
            rows.append(keep)
        if n == 0:
            continue
        for h in range(Hkv):
            k, v = (_meant(s["pool"][i][p, h].flatten(0, 1)[:n], s["scale"][i][p, h].flatten(0, 1)[:n]) for i in range(2))
            for t in range(T):
                if not bool(rows[t].any()):
                    continue
                x = q[b, t, h] @ k[rows[t]].T / math.sqrt(d)
                lse[b, t, h] = torch.logsumexp(x, -1)
                out[b, t, h] = torch.softmax(x, -1) @ v[rows[t]]
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["lse"].shape)}
