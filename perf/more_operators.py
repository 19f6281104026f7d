"""The attention path of a transformer block when serving, as cases to measure:

    write   new tokens' keys and values into a paged cache, in 16 bits or as e4m3 with a scale a token and head
    read    tokens of the cache back as keys and values
    attend  attention of new tokens over the cache: causal, with a sliding window and first tokens that stay visible
    tree    the same for a tree of drafted tokens, each of which sees the cached context and its own ancestors

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it calls
the framework.  ``exact`` computes them in 64 bits.

A sequence's tokens lie in pages [heads, page, dim] of a pool that its row of the table names, and its new tokens
are the last ones: with ``length`` tokens in the cache and ``n`` new, new token i is token length - n + i.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}


def _case(name, op, B, new, length, heads, group, dim, page, dtype, cache, window=0, sinks=0, ragged=False, order="head"):
    c = {"op": op, "B": B, "new": new, "length": length, "heads": heads, "group": group, "dim": dim, "page": page,
         "dtype": dtype, "cache": cache, "window": window, "sinks": sinks, "ragged": ragged, "order": order}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decode step of 48 sequences: one token each, to 8 bits: latency alone
        _case("write_step_e4m3", "write", 48, 1, 500, 8, 4, 128, 64, "bf16", "e4m3", ragged=True),
        # four long prompts, to 8 bits: bandwidth
        _case("write_prompts_e4m3", "write", 4, 8192, 8192, 8, 4, 128, 64, "bf16", "e4m3"),
        # the last tokens of a few sequences of odd lengths and sizes (moved to another cache)
        _case("read_ragged_f16", "read", 9, 301, 777, 5, 3, 96, 24, "f16", "f16", ragged=True),
        # a long shared prefix brought back to 16 bits
        _case("read_prefix_e4m3", "read", 1, 32768, 32768, 8, 4, 128, 64, "bf16", "e4m3"),
        # one token of one sequence of 1200: latency alone
        _case("attend_token_bf16", "attend", 1, 1, 1200, 8, 4, 128, 64, "bf16", "bf16"),
        # a decode step of 64 sequences of up to 8192 tokens in 8 bits: reading the cache
        _case("attend_batch_e4m3", "attend", 64, 1, 8192, 8, 4, 128, 64, "bf16", "e4m3", ragged=True),
        # one token of one long document: the sum is long and there is one row a head
        _case("attend_long_bf16", "attend", 1, 1, 131072, 8, 4, 128, 64, "bf16", "bf16"),
        # a decode step with a window and sinks, small pages, narrow heads
        _case("attend_window_f16", "attend", 100, 1, 16000, 4, 8, 64, 16, "f16", "f16", 1024, 4, ragged=True),
        # a prompt of 8192 tokens: the matrix rate
        _case("attend_prompt_bf16", "attend", 1, 8192, 8192, 8, 4, 128, 64, "bf16", "bf16"),
        # chunks of prompts with odd lengths over what is cached in 8 bits, a window and sinks, an odd group
        _case("attend_chunks_f16", "attend", 5, 1999, 9001, 4, 7, 96, 32, "f16", "e4m3", 1500, 5, ragged=True),
        # drafted trees of 26 tokens
        _case("tree_step_bf16", "tree", 8, 26, 3001, 8, 4, 128, 64, "bf16", "bf16", ragged=True),
        # larger trees for a whole batch, in 8 bits, with a window
        _case("tree_batch_e4m3", "tree", 32, 64, 8000, 8, 4, 128, 64, "bf16", "e4m3", 4096, 4, ragged=True),
    ]


def _size(rng, lo, hi):
    """lo..hi, even over the logarithm; three in ten whole multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.3:
        v = v // 64 * 64
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "tree"))
    while True:
        heads, group = rng.choice((1, 2, 3, 4, 5, 8, 16)), rng.choice((1, 2, 3, 4, 5, 7, 8))
        dim, page = rng.choice((64, 80, 96, 128, 128, 192, 256)), rng.choice((16, 16, 32, 64, 64, 128, 24, 50))
        B = _size(rng, 1, 128)
        length = _size(rng, 1, 65536)
        if op == "tree":
            new = _size(rng, 2, 100)
        elif op == "attend" and rng.random() < 0.5:
            new = 1
        else:
            new = _size(rng, 1, 8192)
        if new > length or B * length * heads * dim > 2 ** 28 or heads * group > 64:
            continue
        if op in ("attend", "tree"):
            dtype = rng.choice(("f16", "bf16"))
            cache = rng.choice((dtype, "e4m3"))
        else:
            dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
            cache = rng.choice(("f16", "bf16", "e4m3")) if dtype == "f32" or op == "read" else rng.choice((dtype, "e4m3"))
        windowed = op in ("attend", "tree") and rng.random() < 0.4
        c = _case(None, op, B, new, length, heads, group, dim, page, dtype, cache, _size(rng, 1, 8192) if windowed else 0,
                  rng.choice((0, 1, 4, 17)) if windowed else 0, rng.random() < 0.7, rng.choice(("head", "head", "token")))
        if work(c)["flops"] <= 5e11:
            return c


def _lengths(case):
    """Every sequence's length and its count of new tokens: the sizes are the case's, whatever the seed."""
    rng = random.Random(case["B"] * 1000003 + case["length"])
    out = []
    for b in range(case["B"]):
        length, new = case["length"], case["new"]
        if case["ragged"] and b:
            if case["op"] != "tree" and new > 1:
                new = rng.randint(1, new)
            length = rng.randint(max(new, length // 4), length)
        out.append((length, new))
    return out


def _seen(length, new, window, sinks):
    """Keys that `new` last tokens of `length` see, as a sum over the tokens, and their union."""
    if not window:
        return new * (length - new) + new * (new + 1) // 2, length
    total = 0
    for i in range(length - new, length):
        low = max(0, i - window + 1)
        total += i - low + 1 + min(sinks, low)
    low = max(0, length - new - window + 1)
    return total, length - low + min(sinks, low)


def work(case):
    e, ce, h, d = SIZE[case["dtype"]], SIZE[case["cache"]], case["heads"], case["dim"]
    row = 2 * (d * ce + (4 if case["cache"] == "e4m3" else 0))  # a token's key and value, in one head
    tokens = sum(n for _, n in _lengths(case))
    if case["op"] in ("write", "read"):
        return {"bytes": tokens * h * (row + 2 * d * e), "flops": 2 * tokens * h * d}
    pairs = keys = 0
    for length, n in _lengths(case):
        if case["op"] == "tree":  # a node sees the context, some ancestors and itself
            p, k = _seen(length - n + 1, 1, case["window"], case["sinks"])
            p, k = p * n, k + n - 1
        else:
            p, k = _seen(length, n, case["window"], case["sinks"])
        pairs, keys = pairs + p, keys + k
    g = case["group"]
    return {"bytes": keys * h * row + 2 * tokens * h * g * d * e, "flops": 4 * pairs * h * g * d}


# ------------------------------------------------------------------ inputs --
def _scale_of(a):
    """The power of two by which a row whose largest value is a fits e4m3 (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(a.clamp_min(2.0 ** -100))
    return torch.ldexp(torch.ones_like(a), e - 9 + (m > 0.875).to(e.dtype))


def _to_e4m3(v):
    a = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax(dim=-1)
    s = _scale_of(a)
    return (v / s[..., None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, ct = DT[case["dtype"]], DT[case["cache"]]
    B, h, d, page = case["B"], case["heads"], case["dim"], case["page"]
    lengths = _lengths(case)
    width = (case["length"] + page - 1) // page
    pages = B * width + 3  # a few that no sequence has

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def pool():
        # what the cache holds already: other tokens' rows, of unit size
        shape = (pages, h, page, d) if case["order"] == "head" else (pages, page, h, d)
        if case["cache"] != "e4m3":
            t, s = normal(*shape).to(ct), None
        else:
            t = torch.empty(shape, dtype=ct, device="cuda")
            s = torch.empty(shape[:3], device="cuda")
            for i in range(0, pages, 1024):
                t[i:i + 1024], s[i:i + 1024] = _to_e4m3(normal(*t[i:i + 1024].shape))
        if case["order"] != "head":
            t, s = t.transpose(1, 2), None if s is None else s.transpose(1, 2)
        return t, s

    s = {"case": case}
    s["k"], s["k_scale"] = pool()
    s["v"], s["v_scale"] = pool()
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[:B * width].view(B, width).to(torch.int32)
    s["lens"] = torch.tensor([n for n, _ in lengths], dtype=torch.int32, device="cuda")
    starts = [0]
    for _, n in lengths:
        starts.append(starts[-1] + n)
    s["tokens"] = T = starts[-1]
    # sequences with equal counts of new tokens need no starts
    s["starts"] = None if T == B * lengths[0][1] else torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["longest"] = case["length"]
    if case["op"] == "write":
        # slices of the rows that a block's fused projection gives; a few channels are much larger than the rest
        big = 1.0 + 9.0 * (torch.rand(h * d, generator=g, device="cuda") < 0.02).float()
        x = torch.cat([normal(T, h * d) * big, normal(T, h * d)], dim=1).to(dt)
        s["new_k"], s["new_v"] = x[:, :h * d].view(T, h, d), x[:, h * d:].view(T, h, d)
    elif case["op"] in ("attend", "tree"):
        s["q"] = normal(T, h * case["group"], d, std=1.5).to(dt)
    if case["op"] == "tree":
        s["tree"] = _trees(B, case["new"], seed)
    if own:
        s["cache"] = _convtile().KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


def _trees(B, n, seed):
    """Random trees of n nodes, as rows of bits: bit j of row i is set where node i sees node j (itself among them)."""
    g = torch.Generator()
    g.manual_seed(seed)
    sees = torch.zeros(B, n, n, dtype=torch.bool)
    every = torch.arange(B)
    for i in range(n):
        if i:
            # a parent among the last few nodes, or the cached context itself
            parent = i - 1 - torch.randint(0, min(i, 8) + 1, (B,), generator=g)
            has = parent >= 0
            sees[every[has], i] = sees[every[has], parent[has]]
        sees[:, i, i] = True
    words = (n + 63) // 64
    bits = torch.zeros(B, n, words * 64, dtype=torch.int64)
    bits[:, :, :n] = sees.to(torch.int64)
    weights = torch.ones(64, dtype=torch.int64) << torch.arange(64)
    return (bits.view(B * n, words, 64) * weights).sum(dim=2).cuda()


# -------------------------------------------------------------- plain forms --
def _places(s):
    """Of every new token: its sequence, its place there, and its page and place in the page."""
    B, T, page = s["case"]["B"], s["tokens"], s["case"]["page"]
    t = torch.arange(T, device="cuda")
    if s["starts"] is None:
        n = T // B
        b = t // n
        at = s["lens"].long()[b] - n + t % n
    else:
        st = s["starts"].long()
        b = torch.searchsorted(st, t, right=True) - 1
        at = s["lens"].long()[b] - (st[b + 1] - t)
    return b, at, s["table"].long()[b, at // page], at % page


def _rows(pool, scale, pages, places=None):
    """Rows of a pool as 32-bit values: of whole pages, or of places in them."""
    if places is None:
        r = pool[pages].float()
        return r if scale is None else r * scale[pages][..., None]
    r = pool[pages, :, places].float()
    return r if scale is None else r * scale[pages, :, places][..., None]


def _plain_write(s):
    _, _, pages, places = _places(s)
    out = {}
    for name in ("k", "v"):
        x = s["new_" + name].float()
        if s["k_scale"] is None:
            s[name][pages, :, places] = x.to(s[name].dtype)
        else:
            q, scale = _to_e4m3(x)
            s[name].view(torch.uint8)[pages, :, places] = q.view(torch.uint8)
            s[name + "_scale"][pages, :, places] = scale
    return _cache_of(s)


def _cache_of(s):
    names = ("k", "v") if s["k_scale"] is None else ("k", "v", "k_scale", "v_scale")
    return {n: s[n] for n in names}


def _plain_read(s):
    _, _, pages, places = _places(s)
    dt = DT[s["case"]["dtype"]]
    return {n: _rows(s[n], s[n + "_scale"], pages, places).to(dt) for n in ("k", "v")}


def _visible(s, at, n, length, tree, keys):
    """[sequences, new tokens, keys]: which keys the new tokens see (at: the first new token's place, [sequences])."""
    c = s["case"]
    k = torch.arange(keys, device="cuda")
    if tree is None:
        place = at[:, None] + torch.arange(n, device="cuda")
        see = (k <= place[..., None]) & (k < length[:, None, None])
        kpos = k.expand(see.shape)
    else:
        # nodes that a node sees come in order behind the context, itself the last
        shift = torch.arange(64, device="cuda")
        bits = ((tree[..., None] >> shift) & 1).flatten(2)[..., :n]
        place = at[:, None] + bits.sum(dim=2) - 1
        rank = bits.cumsum(dim=2) - 1
        node = k[None, :] - at[:, None]
        inside = (node >= 0) & (node < n)
        pick = node.clamp(0, n - 1)[:, None, :].expand(-1, n, -1)
        see = torch.where(inside[:, None, :], bits.gather(2, pick) > 0, (node < 0)[:, None, :])
        kpos = torch.where(inside[:, None, :], at[:, None, None] + rank.gather(2, pick), k[None, None, :])
    if c["window"]:
        see = see & ((kpos > place[..., None] - c["window"]) | (kpos < c["sinks"]))
    return see


def _plain_attend(s):
    c = s["case"]
    B, h, g, d, page = c["B"], c["heads"], c["group"], c["dim"], c["page"]
    out = torch.empty_like(s["q"])
    lengths = _lengths(c)
    if s["starts"] is None:  # sequences with equal counts of new tokens, as many at a time as memory likes
        n = s["tokens"] // B
        many = max(1, min(B, 2 ** 30 // max(1, c["length"] * h * max(d, g * n))))
        groups = [(b, min(B, b + many), b * n, n, c["length"]) for b in range(0, B, many)]
    else:
        groups, t = [], 0
        for b, (length, n) in enumerate(lengths):
            groups.append((b, b + 1, t, n, length))
            t += n
    for b0, b1, t0, n, longest in groups:
        nb = b1 - b0
        width = (longest + page - 1) // page
        keys = width * page
        pages = s["table"][b0:b1, :width].long()
        length = s["lens"][b0:b1].long()
        some = max(1, min(n, 2 ** 29 // max(1, nb * h * g * keys)))  # new tokens at a time
        k = _rows(s["k"], s["k_scale"], pages).permute(0, 2, 4, 1, 3).reshape(nb * h, d, keys)
        v = _rows(s["v"], s["v_scale"], pages).permute(0, 2, 1, 3, 4).reshape(nb * h, keys, d)
        q = s["q"][t0:t0 + nb * n].view(nb, n, h, g, d)
        tree = s["tree"][t0:t0 + nb * n].view(nb, n, -1) if c["op"] == "tree" else None
        if tree is not None:
            some = n
        for i in range(0, n, some):
            m = min(some, n - i)
            see = _visible(s, length - n + i, m, length, tree, keys)
            x = q[:, i:i + m].permute(0, 2, 3, 1, 4).reshape(nb * h, g * m, d).float()
            z = torch.bmm(x, k).mul_(d ** -0.5).view(nb, h, g, m, keys)
            z.masked_fill_(~see[:, None, None], float("-inf"))
            z.sub_(z.amax(dim=-1, keepdim=True)).exp_()
            total = z.sum(dim=-1, keepdim=True)
            y = torch.bmm(z.view(nb * h, g * m, keys), v).view(nb, h, g, m, d) / total
            out[t0:t0 + nb * n].view(nb, n, h, g, d)[:, i:i + m] = y.permute(0, 3, 1, 2, 4).to(out.dtype)
    return {"y": out}


def _plain(s):
    op = s["case"]["op"]
    return _plain_write(s) if op == "write" else _plain_read(s) if op == "read" else _plain_attend(s)


# ------------------------------------------------------------ the framework --
_ct = None


def _convtile():
    global _ct
    if _ct is None:
        from tensor_compiler_tiling_amd import convtile

        _ct = convtile
    return _ct


def _framework(s):
    ct, c = _convtile(), s["case"]
    if c["op"] == "write":
        ct.kv_write(s["cache"], s["new_k"], s["new_v"], s["lens"], table=s["table"], starts=s["starts"])
        return _cache_of(s)
    if c["op"] == "read":
        k, v = ct.kv_read(s["cache"], s["tokens"], s["lens"], table=s["table"], starts=s["starts"], dtype=DT[c["dtype"]])
        return {"k": k, "v": v}
    y = ct.kv_attention(s["q"], s["cache"], s["lens"], table=s["table"], starts=s["starts"], max_len=s["longest"],
                        window=c["window"], sinks=c["sinks"], tree=s.get("tree"))
    return {"y": y}


def run(state):
    return _framework(state) if own else _plain(state)


# -------------------------------------------------------------- definitions --
def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time; an 8-bit cache's written rows before their rounding to 8 bits."""
    s = prepare(case, seed)
    page, h, g, d = case["page"], case["heads"], case["group"], case["dim"]
    lengths = _lengths(case)
    if case["op"] == "write":
        out = {n: t.double().contiguous() for n, t in _cache_of(s).items()}
        t = 0
        for b, (length, n) in enumerate(lengths):
            at = torch.arange(length - n, length, device="cuda")
            where = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
            for name in ("k", "v"):
                x = s["new_" + name][t:t + n].double()
                if case["cache"] == "e4m3":
                    top = x.abs().max(dim=2).values.clamp(min=2.0 ** -100)
                    scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
                    # log2 may be off by a step next to a whole number
                    scale = torch.where(top > 448.0 * scale, 2.0 * scale, scale)
                    scale = torch.where(top <= 224.0 * scale, 0.5 * scale, scale)
                    out[name + "_scale"][where, :, at % page] = scale
                    x = x / scale.unsqueeze(2)
                out[name][where, :, at % page] = x
            t += n
        return out

    def held(name, b, first, last):
        at = torch.arange(first, last, device="cuda")
        where, place = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")], at % page
        x = s[name][where, :, place].double()
        return x if case["cache"] != "e4m3" else x * s[name + "_scale"][where, :, place].double().unsqueeze(2)

    if case["op"] == "read":
        return {name: torch.cat([held(name, b, length - n, length) for b, (length, n) in enumerate(lengths)])
                for name in ("k", "v")}
    out = torch.empty(s["tokens"], h * g, d, dtype=torch.float64, device="cuda")
    t = 0
    for b, (length, n) in enumerate(lengths):
        k, v = held("k", b, 0, length), held("v", b, 0, length)
        ctx = length - n
        step = n if case["op"] == "tree" else max(1, min(n, 2 ** 27 // (g * length)))
        for i in range(0, n, step):
            m = min(step, n - i)
            hidden = torch.zeros(m, length, dtype=torch.bool, device="cuda")
            if case["op"] == "tree":
                rows = [sum((int(w) & (2 ** 64 - 1)) << (64 * j) for j, w in enumerate(r)) for r in s["tree"][t:t + n].tolist()]
                place = torch.empty(n, length, dtype=torch.int64)
                place[:, :ctx] = torch.arange(ctx)
                last = []
                dark = torch.zeros(n, n, dtype=torch.bool)
                for r, word in enumerate(rows):
                    p = ctx
                    for j in range(n):
                        dark[r, j] = not word >> j & 1
                        place[r, ctx + j] = p
                        p += word >> j & 1
                    last.append(p - 1)
                hidden[:, ctx:] = dark.cuda()
                place, own_place = place.cuda(), torch.tensor(last, device="cuda").unsqueeze(1)
            else:
                place = torch.arange(length, device="cuda").unsqueeze(0)
                own_place = torch.arange(ctx + i, ctx + i + m, device="cuda").unsqueeze(1)
                hidden |= place > own_place
            if case["window"]:
                hidden |= (own_place - place >= case["window"]) & (place >= case["sinks"])
            for j in range(h):
                x = s["q"][t + i:t + i + m, j * g:(j + 1) * g].double().reshape(m * g, d)
                z = torch.matmul(x, k[:, j].t().contiguous()).div_(math.sqrt(d)).view(m, g, length)
                z.masked_fill_(hidden.unsqueeze(1), -math.inf)
                y = torch.matmul(torch.softmax(z, dim=2).view(m * g, length), v[:, j].contiguous())
                out[t + i:t + i + m, j * g:(j + 1) * g] = y.view(m, g, d)
        t += n
    return {"y": out}
