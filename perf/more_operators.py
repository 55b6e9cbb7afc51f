"""The operators of a step that checks trees of drafted tokens, and rotary positions with several axes,
as measured cases: positions (time, height, width) of image and video tokens, the plan of a tree, attention
of its nodes over the 4-bit cache, what is accepted of it, and the accepted rows' move in the cache.

``run`` computes each operator in its plain form (elementary torch operations in fp32, in fp64 where angles
of far positions need it), or, with ``own`` set, through the package's entry points.  ``exact`` computes the
same outputs from the definitions in fp64, request by request."""
import math

import torch

own = False

DEV = "cuda"
GROUP = 16  # values of a head that share one e4m3 scale in the cache


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # queries and keys of one step that checks 8 requests' drafts of 8: only latency counts
        dict(name="axes_nodes_t64", op="axes", layout="tokens", b=1, hq=32, hk=8, n=64, d=128, r=128,
             axes=3, cycled=False, interleaved=False, inverse=False, start=100000),
        # the gradients of q and k of a training step on video, B2 H32 N8192 d128
        dict(name="axes_bwd_b2h32n8192d128", op="axes", layout="heads", b=2, hq=32, hk=32, n=8192,
             d=128, r=128, axes=3, cycled=True, interleaved=False, inverse=True, start=1000),
        # a step of 8 requests with 8 drafted tokens behind the last chosen one
        dict(name="plan_b8n9", op="plan", b=8, nodes=9, spread=4, maxlen=8192),
        # a large batch of ragged trees of up to 64 nodes
        dict(name="plan_b1000n64", op="plan", b=1000, nodes=64, spread=16, maxlen=16384),
        # one request, a short cache, no shared heads, a small tree
        dict(name="attend_one_short", op="attend", b=1, hq=16, hk=16, d=64, page=16, minlen=200,
             maxlen=256, nodes=9, spread=4),
        # a serving batch: 64 ragged requests with trees of up to 16 nodes, 4 query heads to a key head
        dict(name="attend_b64n16", op="attend", b=64, hq=32, hk=8, d=128, page=64, minlen=500, maxlen=8192,
             nodes=16, spread=6),
        # larger trees, an odd number of nodes and of heads in a group
        dict(name="attend_b16n41", op="attend", b=16, hq=24, hk=8, d=128, page=32, minlen=1000,
             maxlen=16384, nodes=41, spread=10),
        # one long request with a wide tree: the work has to be split along the cache
        dict(name="attend_long_b1n60", op="attend", b=1, hq=32, hk=4, d=128, page=128, minlen=262000,
             maxlen=262144, nodes=60, spread=16),
        # what 8 requests accept of their trees
        dict(name="accept_b8n9", op="accept", b=8, nodes=9, spread=4, page=64, maxlen=8192),
        # a large batch, some requests refused or ended, pages given back
        dict(name="accept_b1000n64", op="accept", b=1000, nodes=64, spread=16, page=16, maxlen=4096),
        # accepted rows of 8 requests to their places, in the caches of 4 layers
        dict(name="move_b8l4", op="move", b=8, nodes=9, layers=4, h=8, d=128, page=64, pages=64),
        # 64 requests with larger trees, 64 layers
        dict(name="move_b64l64", op="move", b=64, nodes=41, layers=64, h=8, d=128, page=32, pages=512),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "axes", "plan", "attend", "attend", "attend", "attend", "accept", "move"])
    d = rng.choice([64, 128])
    if op == "axes":
        r = d if rng.random() < 0.5 else 16 * rng.randint(1, d // 16)
        common = dict(op=op, d=d, r=r, axes=rng.choice([2, 3, 3, 4]), cycled=rng.random() < 0.5,
                      interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5)
        if rng.random() < 0.5:
            return dict(common, layout="tokens", b=1, hq=rng.choice([8, 16, 32, 40]),
                        hk=rng.choice([1, 2, 8]), n=_spread(rng, 1, 20000), start=_spread(rng, 1000, 1000000))
        h = rng.choice([2, 8, 16, 32])
        return dict(common, layout="heads", b=rng.randint(1, 2), hq=h, hk=h, n=_spread(rng, 100, 8192), start=0)
    if op == "plan":
        n = _spread(rng, 2, 255)
        return dict(op=op, b=_spread(rng, 1, 60000 // n if n > 64 else 1000), nodes=n, spread=_spread(rng, 1, 32),
                    maxlen=_spread(rng, 300, 16384))
    if op == "accept":
        n = _spread(rng, 2, 128)
        return dict(op=op, b=_spread(rng, 1, 60000 // n if n > 64 else 1000), nodes=n, spread=_spread(rng, 1, 32),
                    page=rng.choice([16, 32, 64, 128]), maxlen=_spread(rng, 300, 4096))
    if op == "move":
        n = _spread(rng, 4, 128)
        page, b = rng.choice([16, 32, 64, 128]), _spread(rng, 1, 64)
        return dict(op=op, b=b, nodes=n, layers=_spread(rng, 1, 64), h=rng.choice([1, 2, 4, 8]), d=d, page=page,
                    pages=b * (-(-n // page) + 1) + 5)
    hk = rng.choice([1, 2, 4, 8])
    common = dict(op=op, hq=hk * rng.choice([1, 2, 3, 4, 5]), hk=hk, d=d, page=rng.choice([16, 32, 64, 128]),
                  spread=_spread(rng, 1, 32))
    kind = rng.choice(["batch", "batch", "batch", "long", "wide"])
    if kind == "long":
        top = _spread(rng, 16384, 131072)
        return dict(common, b=rng.randint(1, 2), minlen=top // 2, maxlen=top, nodes=_spread(rng, 2, 60))
    if kind == "wide":
        top = _spread(rng, 500, 4096)
        return dict(common, b=rng.randint(1, 3), minlen=top // 2, maxlen=top, nodes=_spread(rng, 60, 255))
    top = _spread(rng, 60, 8192)
    return dict(common, b=_spread(rng, 1, 32), minlen=max(1, top // 8), maxlen=top, nodes=_spread(rng, 2, 50))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _page_bytes(page, d):
    return page * (d // 2 + d // GROUP)


def _sections(pairs, axes):
    """Pairs of each axis: a smaller first one (time) and nearly equal others."""
    if axes == 2:
        return [pairs - pairs // 2, pairs // 2]
    first = pairs // (axes + 1)
    rest = pairs - first
    more = [rest // (axes - 1)] * (axes - 1)
    more[0] += rest - sum(more)
    return [first] + more


def _pair_axes(pairs, axes, cycled):
    """The axis of each pair: one section behind the other, or the axes in turn until theirs are used up."""
    left = _sections(pairs, axes)
    if not cycled:
        return torch.tensor([a for a, n in enumerate(left) for _ in range(n)], dtype=torch.uint8, device=DEV)
    out = []
    while len(out) < pairs:
        for a in range(axes):
            if left[a] > 0:
                left[a] -= 1
                out.append(a)
    return torch.tensor(out, dtype=torch.uint8, device=DEV)


def _video_positions(n, axes, at):
    """Some text, then frames of a square grid: [axes, n], from position `at` (a tensor) on."""
    i = torch.arange(n, device=DEV)
    text, side = n // 8, max(2, math.isqrt(n) // 2)
    j = (i - text).clamp(min=0)
    grid = [j // (side * side), j // side % side, j % side, (j // 7) % 5]
    return torch.stack([torch.where(i < text, i, text + g) for g in grid[:axes]]).int() + at


def _tree(b, nodes, spread, host, g, whole=False):
    """Ragged trees: nodes of each request (they belong to the case: they set the outputs' shapes), offsets,
    and each node's parent among its request's nodes, -1 for the first."""
    count = torch.randint(max(1, nodes // 2), nodes + 1, (b,), generator=host)
    count[0] = nodes
    off = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])
    total = int(off[-1])
    off = off.to(DEV)
    t = torch.arange(total, device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[r]
    u = torch.rand(total, device=DEV, generator=g)
    parents = i - 1 - (u * u * i.clamp(max=spread)).long()
    return off.int(), torch.where(i > 0, parents.clamp(min=0), -1).int()


def _fill_cache(cache, page, d, g):
    """Normal keys and values with a few large channels, quantised into every page."""
    pages, h = cache.shape[:2]
    loud = 1 + 4 * (torch.rand(h, 1, 1, d, device=DEV, generator=g) < 0.03)
    for p in range(0, pages, max(1, pages // 8)):
        part = cache[p:p + max(1, pages // 8)]
        x = torch.randn(part.shape[0], h, 2, page, d, device=DEV, generator=g) * loud
        x = x.unflatten(-1, (-1, GROUP))
        s = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        t = x / s.float()[..., None]
        a = t.abs()
        code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
                + (a > 5.0)) | (torch.signbit(t).to(torch.uint8) << 3)
        code = code.flatten(-2)
        part[..., :page * d // 2].unflatten(-1, (page, d // 2)).copy_(code[..., 0::2] | (code[..., 1::2] << 4))
        part[..., page * d // 2:].unflatten(-1, (page, d // GROUP)).copy_(s.view(torch.uint8))


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    c = dict(case)
    op = c["op"]
    normal = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, device=DEV, generator=g, dtype=torch.int32)  # noqa: E731
    host = torch.Generator().manual_seed(5)
    st = {"op": op, "case": c}
    if op == "axes":
        n, pairs = c["n"], c["r"] // 2
        st["freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
        st["turns"] = (st["freq"] * (2.0 ** 64 / (2 * math.pi))).round().to(torch.int64)
        st["axes"] = _pair_axes(pairs, c["axes"], c["cycled"])
        at = ints(0, c["start"] + 1, 1) if c["start"] else 0
        st["positions"] = _video_positions(n, c["axes"], at).contiguous()
        if c["layout"] == "tokens":
            # rows of a projection that makes queries and keys side by side
            both = normal(n, c["hq"] + c["hk"], c["d"])
            st["q"], st["k"] = both[:, :c["hq"]], both[:, c["hq"]:]
        else:
            st["q"], st["k"] = normal(c["b"], c["hq"], n, c["d"]), normal(c["b"], c["hk"], n, c["d"])
        return st
    if op == "move":
        b, n, page = c["b"], c["nodes"], c["page"]
        count = torch.randint(1, max(1, min(n // 3, 7)) + 1, (b,), generator=host)
        st["cache"] = torch.randint(0, 256, (c["layers"], c["pages"], c["h"], 2, _page_bytes(page, c["d"])),
                                    device=DEV, generator=g, dtype=torch.uint8)
        st["layers"] = list(st["cache"].unbind(0))
        # each request's n rows lie in consecutive places of its pages, from anywhere in the first one
        width = -(-n // page) + 1
        pages = torch.randperm(c["pages"], device=DEV, generator=g)[:b * width].view(b, width)
        place = ints(0, page, b, 1) + torch.arange(n, device=DEV)
        slots = pages.gather(1, place // page) * page + place % page
        # the accepted nodes of a request, in their order; all behind the places that they go to
        rank = torch.rand(b, n, device=DEV, generator=g)
        rank[:, :8] = 2.0
        picked = rank.argsort(1)[:, :8].sort(1).values  # of n - 8 or more nodes
        i = torch.arange(n, device=DEV)
        moved = i[None] < count.to(DEV)[:, None]
        source = torch.where(moved[:, :8], slots.gather(1, picked)[:, :moved[:, :8].shape[1]], -1) if n >= 16 else \
            torch.where(moved, slots.flip(1), -1)
        full = torch.full_like(slots, -1)
        full[:, :source.shape[1]] = source
        st["slots"], st["sources"] = slots.reshape(-1).int(), full.reshape(-1).int()
        st["q_offsets"] = (torch.arange(b + 1, device=DEV) * n).int()
        st["counts"] = count.to(DEV).int()
        st["moves"] = [(moved & (full >= 0)).reshape(-1).nonzero().reshape(-1)]
        return st
    off, parents = _tree(c["b"], c["nodes"], c["spread"], host, g)
    st["q_offsets"], st["parents"] = off, parents
    total, b = parents.numel(), c["b"]
    count = off[1:] - off[:-1]
    if op == "plan":
        st["lens"] = ints(1, c["maxlen"], b)
        return st
    st["words"] = -(-c["nodes"] // 32)
    st["seen"] = _plain_plan(st, torch.zeros(b, device=DEV))[1]
    page = c["page"]
    if op == "attend":
        width = -(-c["maxlen"] // page)
        st["lens"] = torch.maximum(ints(c["minlen"], c["maxlen"] + 1, b), count.clamp(max=width * page))
        st["q"] = normal(total, c["hq"], c["d"]) * 2
        st["table"] = torch.randperm(b * width, device=DEV, generator=g).int().view(b, width)
        st["cache"] = torch.empty(b * width, c["hk"], 2, _page_bytes(page, c["d"]), dtype=torch.uint8, device=DEV)
        _fill_cache(st["cache"], page, c["d"], g)
        st["scale"] = 1.0 / math.sqrt(c["d"])
        return st
    # accept: what page planning left of the step before, and what the model chose at each node
    width = -(-(c["maxlen"] + c["nodes"]) // page)
    lens = ints(1, c["maxlen"] + 1, b)
    refused = torch.rand(b, device=DEV, generator=g) < (0.05 if b > 8 else 0.0)
    after = torch.where(refused, lens, lens + count)
    r = torch.repeat_interleave(torch.arange(b, device=DEV), count.long(), output_size=total)
    i = torch.arange(total, device=DEV) - off[r]
    st["table"] = torch.randperm(b * width, device=DEV, generator=g).int().view(b, width)
    place = (lens[r] + i).long()
    slots = st["table"][r, place // page] * page + (place % page).int()
    st["slots"] = torch.where(refused[r], -1, slots).int()
    st["lens"], st["lens_after"] = lens, after
    have = (after + page - 1) // page
    spare = torch.arange(width, device=DEV)[None] >= have[:, None]
    free = spare.sum().int()
    st["queue"] = st["table"].reshape(-1)[torch.sort(spare.reshape(-1).to(torch.int8), descending=True,
                                                     stable=True).indices].roll(5 % (b * width)).contiguous()
    st["queue_state"] = torch.stack([torch.full_like(free, 5 % (b * width)), free])
    # tokens of a vocabulary of 32000; at most nodes the model chose what one of the children holds
    tokens, choices = ints(0, 32000, total), ints(0, 32000, total)
    child = torch.arange(total, device=DEV, dtype=torch.int64)
    child = torch.where((torch.rand(total, device=DEV, generator=g) < 0.8) & (parents >= 0), child, -1)
    taken = torch.full((total,), -1, dtype=torch.int64, device=DEV)
    taken.scatter_reduce_(0, (off[r] + parents.clamp(min=0)).long(), child, "amax")
    st["tokens"], st["choices"] = tokens, torch.where(taken >= 0, tokens[taken.clamp(min=0)], choices)
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _plain_axes(x, st):
    c = st["case"]
    r = c["r"]
    at = st["positions"].double()[st["axes"].long()]  # [pairs, n]
    angle = at.T * st["freq"]
    angle = -angle if c["inverse"] else angle
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["layout"] == "tokens":
        cos, sin = cos[:, None], sin[:, None]
    xf = x.float()
    a, b = (xf[..., 0:r:2], xf[..., 1:r:2]) if c["interleaved"] else (xf[..., :r // 2], xf[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([y, z], -1).flatten(-2) if c["interleaved"] else torch.cat([y, z], -1)
    return torch.cat([y, xf[..., r:]], -1).to(x.dtype)


def _padded(st, x, fill):
    """Packed values of nodes as [b, nodes], and each packed node's request and number."""
    off, n = st["q_offsets"].long(), st["case"]["nodes"]
    t = torch.arange(x.numel(), device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[r]
    out = torch.full((off.numel() - 1, n), fill, dtype=torch.int64, device=DEV)
    out[r, i] = x.long()
    return out, r, i


def _plain_plan(st, lens):
    n = st["case"]["nodes"]
    up, r, i = _padded(st, st["parents"], -1)
    node = torch.arange(n, device=DEV)
    step = (up[:, :, None] == node).float() + torch.eye(n, device=DEV)  # a node and its parent
    for _ in range(max(1, math.ceil(math.log2(n)))):  # of ever more generations
        step = (step @ step).clamp(max=1)
    seen = step.bool()[r, i]
    words = -(-n // 32)
    bits = torch.zeros(seen.shape[0], 32 * words, dtype=torch.int64, device=DEV)
    bits[:, :n] = seen
    word = (bits.unflatten(1, (words, 32)) << torch.arange(32, device=DEV)).sum(-1)
    word = torch.where(word >= 1 << 31, word - (1 << 32), word)
    return [(lens[r] + seen.sum(-1) - 1).int(), word.int()]


def _bits(seen):
    """[T, words] of int32 as truth values [T, 32 words]."""
    return ((seen[..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).bool().flatten(-2)


def _plain_attend(st):
    c = st["case"]
    page, hk, d, n = c["page"], c["hk"], c["d"], c["nodes"]
    b, width = st["table"].shape
    cache, rows = st["cache"], st["table"].long()
    codes = cache[..., :page * d // 2].unflatten(-1, (page, d // 2))[rows]
    scales = cache[..., page * d // 2:].unflatten(-1, (page, d // GROUP))[rows]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    grid = torch.cat([grid, -grid])
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    kv = (grid[code].unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)
    del code
    kv = kv.permute(3, 0, 2, 1, 4, 5).flatten(3, 4)  # [b, width, hk, 2, page, d] -> [2, b, hk, keys, d]
    lens, off = st["lens"].long(), st["q_offsets"].long()
    t = torch.arange(st["q"].shape[0], device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[r]
    q = torch.zeros(b, n, c["hq"], d, device=DEV)
    q[r, i] = st["q"].float()
    bits = torch.zeros(b, n, 32 * st["words"], dtype=torch.bool, device=DEV)
    bits[r, i] = _bits(st["seen"])
    # keys before the tree are seen by all its nodes, those of the tree as the bits say
    j = torch.arange(width * page, device=DEV)[None] - (lens - (off[1:] - off[:-1]))[:, None]
    at = j.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, n, -1)
    seen = torch.where((j < 0)[:, None], True, bits.gather(2, at))
    seen &= (j < (off[1:] - off[:-1])[:, None])[:, None]
    q = q.permute(0, 2, 1, 3).reshape(b, hk, -1, d)  # heads of one key head side by side
    x = (q @ kv[0].transpose(-1, -2)) * st["scale"]
    x = x.unflatten(2, (-1, n)).masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ kv[1]).unflatten(2, (-1, n)) / total.clamp(min=1e-38)
    lse = (m + torch.log(total)).squeeze(-1)
    o, lse = o.flatten(1, 2).transpose(1, 2), lse.flatten(1, 2).transpose(1, 2)
    return [o[r, i].to(torch.bfloat16), lse[r, i]]


def _plain_accept(st):
    page, n = st["case"]["page"], st["case"]["nodes"]
    up, r, i = _padded(st, st["parents"], -1)
    token, _, _ = _padded(st, st["tokens"], -1)
    choice, _, _ = _padded(st, st["choices"], -2)
    slot, _, _ = _padded(st, st["slots"], -1)
    b = up.shape[0]
    node = torch.arange(n, device=DEV)
    hit = (up >= 0) & (token == choice.gather(1, up.clamp(min=0)))
    # of several children that hold the chosen token the first
    earlier = (up[:, :, None] == up[:, None]) & hit[:, None] & (node[None] < node[:, None])
    good = (hit & ~earlier.any(-1)) | (node == 0)
    seen = torch.zeros(b, n, 32 * st["words"], dtype=torch.bool, device=DEV)
    seen[r, i] = _bits(st["seen"])
    seen = seen[:, :, :n]
    there = torch.zeros_like(good)
    there[r, i] = True
    lens, after = st["lens"].long(), st["lens_after"].long()
    on = there & ~(seen & ~good[:, None]).any(-1) & (after > lens)[:, None]
    count = on.sum(-1)
    place = seen.sum(-1) - 1
    path = torch.full((b, n + 1), -1, dtype=torch.int64, device=DEV)
    path.scatter_(1, torch.where(on, place, n), torch.where(on, node, -1))
    path = path[:, :n]
    source = torch.where(path >= 0, slot.gather(1, path.clamp(min=0)), -1)
    last = path.gather(1, (count - 1).clamp(min=0)[:, None])
    chosen = torch.where(count > 0, choice.gather(1, last.clamp(min=0))[:, 0], -1)
    length = torch.minimum(lens, after) + count
    have, keep = -(-after // page), -(-length // page)
    # pages behind the last one that is kept go behind the free ones, in the requests' order
    back = (have - keep).clamp(min=0)
    queue, table = st["queue"], st["table"]
    cap, width = queue.numel(), table.shape[1]
    head, free = st["queue_state"][0].long(), st["queue_state"][1].long()
    k = torch.arange(width, device=DEV)[None] - keep[:, None]
    at = (head + free + (back.cumsum(0) - back)[:, None] + k) % cap
    at = torch.where((k >= 0) & (k < back[:, None]), at, cap)
    spare = torch.cat([queue, queue[:1]])
    spare[at.reshape(-1)] = table.reshape(-1)
    queue.copy_(spare[:-1])
    state = torch.stack([head, free + back.sum()])
    return [length.int(), count.int(), path[r, i].int(), chosen.int(), source[r, i].int(), state.int(), queue]


def _plain_move(st):
    c = st["case"]
    page, d = c["page"], c["d"]
    cache = st["cache"]
    codes = cache[..., :page * d // 2].unflatten(-1, (page, d // 2))
    scales = cache[..., page * d // 2:].unflatten(-1, (page, d // GROUP))
    at = st["moves"][0]
    src, dst = st["sources"][at].long(), st["slots"][at].long()
    codes[:, dst // page, :, :, dst % page] = codes[:, src // page, :, :, src % page]
    scales[:, dst // page, :, :, dst % page] = scales[:, src // page, :, :, src % page]
    return cache


def run(st):
    c, op = st["case"], st["op"]
    if own:
        import exact_attention_13_gb300 as ea

        if op == "axes":
            return ea.rope_axes(st["q"], st["k"], st["positions"], st["turns"], st["axes"],
                                interleaved=c["interleaved"], inverse=c["inverse"])
        if op == "plan":
            p = ea.tree_plan(st["parents"], st["q_offsets"], st["lens"], max_nodes=c["nodes"])
            return [p.positions, p.seen]
        if op == "attend":
            return ea.kv4_tree_fwd(st["q"], st["cache"], st["table"], st["lens"], st["q_offsets"], st["seen"],
                                   max_q=c["nodes"], scale=st["scale"])
        if op == "accept":
            a = ea.tree_accept(st["parents"], st["seen"], st["tokens"], st["choices"], st["lens"],
                               st["lens_after"], st["q_offsets"], st["slots"], st["table"], st["queue"],
                               st["queue_state"], page_size=c["page"])
            return [a.lens, a.counts, a.path, a.next_tokens, a.sources, a.queue_state, st["queue"]]
        ea.kv4_move(st["layers"], st["sources"], st["slots"], st["q_offsets"], st["counts"], c["d"])
        return st["cache"]
    if op == "axes":
        return (_plain_axes(st["q"], st), _plain_axes(st["k"], st))
    if op == "plan":
        return _plain_plan(st, st["lens"])
    if op == "attend":
        return _plain_attend(st)
    return _plain_accept(st) if op == "accept" else _plain_move(st)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op == "axes":
        n = c["b"] * c["n"] * (c["hq"] + c["hk"])
        return {"bytes": n * c["d"] * 4 + 4 * c["axes"] * c["n"] + 4.5 * c["r"], "flops": 3 * n * c["r"]}
    if op == "move":
        host = torch.Generator().manual_seed(5)
        rows = int(torch.randint(1, max(1, min(c["nodes"] // 3, 7)) + 1, (c["b"],), generator=host).sum())
        row = c["layers"] * c["h"] * 2 * (c["d"] // 2 + c["d"] // GROUP)
        return {"bytes": 2 * rows * row + 8 * rows + 8 * c["b"], "flops": 0}
    host = torch.Generator().manual_seed(5)
    count = torch.randint(max(1, c["nodes"] // 2), c["nodes"] + 1, (c["b"],), generator=host)
    count[0] = c["nodes"]
    total, words = int(count.sum()), -(-c["nodes"] // 32)
    if op == "plan":
        return {"bytes": total * (8 + 4 * words) + 8 * c["b"], "flops": 0}
    if op == "accept":
        # parents, bits, tokens, choices and slots in, path and sources out; a request's lengths and counts
        return {"bytes": total * (24 + 4 * words) + 24 * c["b"], "flops": 0}
    keys = c["b"] * (c["minlen"] + c["maxlen"]) / 2
    cache = keys * c["hk"] * 2 * (c["d"] // 2 + c["d"] // GROUP)
    return {"bytes": cache + total * (c["hq"] * (4 * c["d"] + 4) + 4 * words),
            "flops": 4 * c["d"] * c["hq"] * total * keys / c["b"]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _decode(byte_codes, byte_scales):
    """Values in fp64 from the bit fields of e2m1 codes and e4m3 scales."""
    lo, hi = byte_codes.int() % 16, byte_codes.int() // 16
    n = torch.stack([lo, hi], -1).reshape(*byte_codes.shape[:-1], -1)
    e, m = (n // 2) % 4, (n % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e.double() - 1))
    v = torch.where(n >= 8, -v, v)
    b = byte_scales.int()
    e, m = (b // 8) % 16, (b % 8).double()
    s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7))
    return v * s.repeat_interleave(GROUP, -1)


def _family(parents):
    """Truth values [n, n] of one tree: row i holds node i and the nodes above it."""
    above = torch.zeros(len(parents), len(parents), dtype=torch.bool)
    for i, p in enumerate(parents):
        if p >= 0:
            above[i] = above[p]
        above[i, i] = True
    return above


def exact(case, seed):
    c = case
    if c["op"] in ("plan", "accept", "move"):
        return None  # whole numbers and copied bytes
    st = prepare(case, seed)
    if c["op"] == "axes":
        out = []
        h = c["r"] // 2
        angle = torch.stack([st["positions"][a].double() * f for a, f in zip(st["axes"].tolist(), st["freq"])], -1)
        turn = torch.exp(1j * angle)
        turn = turn.conj() if c["inverse"] else turn
        turn = turn[:, None] if c["layout"] == "tokens" else turn
        for x in (st["q"], st["k"]):
            y = x.double()
            first = slice(0, c["r"], 2) if c["interleaved"] else slice(0, h)
            second = slice(1, c["r"], 2) if c["interleaved"] else slice(h, c["r"])
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return tuple(out)
    page, d, group = c["page"], c["d"], c["hq"] // c["hk"]
    off, parents = st["q_offsets"].tolist(), st["parents"].tolist()
    outs, lses = [], []
    for b, n in enumerate(st["lens"].tolist()):
        blocks = st["cache"][st["table"][b, :-(-n // page)].long()]  # [pages, hk, 2, bytes]
        codes = blocks[..., :page * d // 2].reshape(*blocks.shape[:3], page, -1)
        scales = blocks[..., page * d // 2:].reshape(*blocks.shape[:3], page, -1)
        kv = _decode(codes, scales).permute(2, 1, 0, 3, 4).reshape(2, c["hk"], -1, d)[:, :, :n]
        q = st["q"][off[b]:off[b + 1]].double().transpose(0, 1)  # [hq, nodes, d]
        rows = q.shape[1]
        hidden = ~_family(parents[off[b]:off[b + 1]]).to(DEV)[:, max(0, rows - n):]
        o, lse = torch.empty_like(q), torch.empty_like(q[..., 0])
        for h in range(c["hq"]):
            x = st["scale"] * q[h] @ kv[0, h // group].T
            x[:, max(0, n - rows):].masked_fill_(hidden, -math.inf)
            lse[h] = torch.logsumexp(x, -1)
            o[h] = torch.exp(x - lse[h][:, None].clamp(min=-1e300)) @ kv[1, h // group]
        outs.append(o.transpose(0, 1))
        lses.append(lse.transpose(0, 1))
    return [torch.cat(outs), torch.cat(lses)]
