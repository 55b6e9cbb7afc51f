"""The operators of the serving and training path around attention, as measured cases: rotary
positions, page planning, the 4-bit key/value cache (write and read back) and attention over it.

``run`` computes each operator in its plain form (elementary torch operations in fp32, in fp64
where angles of far positions need it), or, with ``own`` set, through the package's entry points.
``exact`` computes the same outputs from the definitions in fp64, request by request."""
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
        # one decode step of 8 requests: only latency counts
        dict(name="rope_decode_t8", op="rope", layout="tokens", b=1, hq=32, hk=8, n=8, d=128, r=128,
             interleaved=False, inverse=False, scaled=False, pos=131072),
        # q and k of a training step at the headline attention shape (B2 H32 N8192 d128)
        dict(name="rope_fwd_b2h32n8192d128", op="rope", layout="heads", b=2, hq=32, hk=32, n=8192,
             d=128, r=128, interleaved=False, inverse=False, scaled=False, pos=0),
        # gradients of q and k at B4 H16 N2048 d128, interleaved pairs, half of the head rotated,
        # frequencies scaled for a long context
        dict(name="rope_bwd_b4h16n2048d128", op="rope", layout="heads", b=4, hq=16, hk=16, n=2048,
             d=128, r=64, interleaved=True, inverse=True, scaled=True, pos=0),
        # pages of one decode step: 8 requests, one token each
        dict(name="plan_decode_b8", op="plan", b=8, page=64, maxlen=8192, chunk=1, scarce=False),
        # a mixed step of 1000 requests: prompt chunks, decode tokens, finished requests, and not
        # enough free pages for all
        dict(name="plan_mixed_b1000", op="plan", b=1000, page=16, maxlen=16384, chunk=300, scarce=True),
        # one decode step's keys and values of 64 requests into the cache, and read back
        dict(name="append_decode_t64", op="append", t=64, h=8, d=128, page=64, pages=4096),
        # a long prompt chunk, odd length, head dim 64
        dict(name="append_prompt_t8191", op="append", t=8191, h=16, d=64, page=16, pages=4096),
        # the smallest call: one request, one token, a short cache, no shared heads
        dict(name="attend_one_short", op="attend", b=1, hq=16, hk=16, d=64, page=16, minlen=200,
             maxlen=256, q=1, ragged_q=False, causal=True),
        # a decode step of 64 ragged requests, 4 query heads to a key head
        dict(name="attend_decode_b64", op="attend", b=64, hq=32, hk=8, d=128, page=64, minlen=500,
             maxlen=8192, q=1, ragged_q=False, causal=True),
        # one long request: the work has to be split along the cache
        dict(name="attend_long_b1", op="attend", b=1, hq=32, hk=4, d=128, page=128, minlen=262000,
             maxlen=262144, q=1, ragged_q=False, causal=True),
        # a few drafted tokens per request checked at once, odd number of heads in a group
        dict(name="attend_draft_b16", op="attend", b=16, hq=24, hk=8, d=128, page=32, minlen=1000,
             maxlen=16384, q=5, ragged_q=True, causal=True),
        # prompt chunks on top of what the cache holds
        dict(name="attend_chunk_b4", op="attend", b=4, hq=32, hk=8, d=128, page=64, minlen=4096,
             maxlen=8192, q=512, ragged_q=True, causal=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "plan", "append", "attend", "attend", "attend", "attend"])
    d = rng.choice([64, 128])
    if op == "rope":
        r = d if rng.random() < 0.5 else 16 * rng.randint(1, d // 16)
        common = dict(op=op, d=d, r=r, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5,
                      scaled=rng.random() < 0.5)
        if rng.random() < 0.5:
            return dict(common, layout="tokens", b=1, hq=rng.choice([8, 16, 32, 40]),
                        hk=rng.choice([1, 2, 8]), n=_spread(rng, 1, 20000),
                        pos=_spread(rng, 1000, 1000000))
        h, n = rng.choice([2, 8, 16, 32]), _spread(rng, 100, 8192)
        return dict(common, layout="heads", b=rng.randint(1, 2), hq=h, hk=h, n=n, pos=0)
    if op == "plan":
        return dict(op=op, b=_spread(rng, 1, 1500), page=rng.choice([16, 32, 64, 128]),
                    maxlen=_spread(rng, 200, 16384), chunk=_spread(rng, 1, 300),
                    scarce=rng.random() < 0.3)
    if op == "append":
        return dict(op=op, t=_spread(rng, 1, 8192), h=rng.choice([1, 2, 4, 8, 16]), d=d,
                    page=rng.choice([16, 32, 64, 128]), pages=_spread(rng, 600, 4096))
    hk = rng.choice([1, 2, 4, 8])
    kind = rng.choice(["decode", "decode", "draft", "long", "chunk"])
    common = dict(op=op, hq=hk * rng.choice([1, 2, 3, 4, 7, 8]), hk=hk, d=d,
                  page=rng.choice([16, 32, 64, 128]), causal=rng.random() < 0.8)
    if kind == "long":
        top = _spread(rng, 16384, 200000)
        return dict(common, b=rng.randint(1, 2), minlen=top // 2, maxlen=top, q=rng.randint(1, 2),
                    ragged_q=False)
    if kind == "chunk":
        top = _spread(rng, 500, 4096)
        return dict(common, b=rng.randint(1, 3), minlen=top // 2, maxlen=top,
                    q=_spread(rng, 20, 500), ragged_q=True)
    top = _spread(rng, 10, 8192)
    return dict(common, b=_spread(rng, 1, 48), minlen=max(1, top // 8), maxlen=top,
                q=1 if kind == "decode" else rng.randint(2, 8), ragged_q=kind == "draft")


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _frequencies(r, scaled):
    """Angular step per position of each pair (fp64), and the factor on the rotated values."""
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    f = 10000.0 ** (-2.0 * i / r)
    if not scaled:
        return f, 1.0
    # by parts: pairs that turn often within the original context keep their frequency, pairs
    # that turn less than once are slowed down by the factor, a ramp in between
    factor, context, fast, slow = 8.0, 4096, 32.0, 1.0
    at = lambda turns: r * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), r - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _page_bytes(page, d):
    return page * (d // 2 + d // GROUP)


def _fill_cache(cache, page, d, g):
    """Normal keys and values with a few large channels, quantised into every page."""
    pages, h = cache.shape[:2]
    loud = 1 + 4 * (torch.rand(h, 1, 1, d, device=DEV, generator=g) < 0.03)
    for p in range(0, pages, max(1, pages // 8)):
        part = cache[p:p + max(1, pages // 8)]
        x = torch.randn(part.shape[0], h, 2, page, d, device=DEV, generator=g) * loud
        codes, scales = _quantise(x.bfloat16().float())
        part[..., :page * d // 2].unflatten(-1, (page, d // 2)).copy_(codes)
        part[..., page * d // 2:].unflatten(-1, (page, d // GROUP)).copy_(scales)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    c = dict(case)
    op = c["op"]
    normal = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()  # noqa: E731
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, device=DEV, generator=g, dtype=torch.int32)  # noqa: E731
    # how many tokens each request brings belongs to the case: it sets the outputs' shapes
    host = torch.Generator().manual_seed(5)
    st = {"op": op, "case": c}
    if op == "rope":
        freq, mscale = _frequencies(c["r"], c["scaled"])
        # angular steps in units of 2^-64 turn: position * step wraps to the exact part of a turn
        st["freq"], st["mscale"] = freq, mscale
        st["turns"] = (freq * (2.0 ** 64 / (2 * math.pi))).round().to(torch.int64)
        if c["layout"] == "tokens":
            st["q"], st["k"] = normal(c["n"], c["hq"], c["d"]), normal(c["n"], c["hk"], c["d"])
            st["positions"] = ints(0, c["pos"], c["n"])
        else:
            st["q"] = normal(c["b"], c["hq"], c["n"], c["d"])
            st["k"] = normal(c["b"], c["hk"], c["n"], c["d"])
            st["positions"] = torch.arange(c["n"], device=DEV, dtype=torch.int32)
        return st
    if op == "plan":
        b, page, width = c["b"], c["page"], -(-c["maxlen"] // c["page"])
        lens = ints(0, c["maxlen"] + 1, b)
        new = torch.randint(1, c["chunk"] + 1, (b,), generator=host, dtype=torch.int32).to(DEV)
        kind = torch.rand(b, generator=host).to(DEV)
        # some requests finish (-1), some wait (0), most decode one token when chunks are long
        if c["chunk"] > 1:
            new = torch.where(kind < 0.7, torch.ones_like(new), new)
            new = torch.where(kind < 0.1, torch.zeros_like(new), new)
            new = torch.where(kind < 0.05, torch.full_like(new, -1), new)
            lens = torch.where((kind >= 0.7) & (kind < 0.85), torch.zeros_like(lens), lens)
        pages = b * width
        order = torch.randperm(pages, device=DEV, generator=g).int()
        st["table"] = order.view(b, width).contiguous()
        have = (lens + page - 1) // page
        spare = (torch.arange(width, device=DEV)[None] >= have[:, None]).reshape(-1)
        free = order[torch.sort(spare.to(torch.int8), descending=True, stable=True).indices]
        head = 7 % pages
        st["queue"] = torch.roll(free, head).contiguous()
        count = spare.sum().int()
        if c["scarce"]:
            grow = ((lens + new.clamp(min=0) + page - 1) // page - have).clamp(min=0).sum()
            count = torch.minimum(count, (grow * 3) // 4)
        st["queue_state"] = torch.stack([torch.full_like(count, head), count]).int()
        st["lens"], st["new"] = lens, new
        st["tokens"] = int(new.clamp(min=0).sum()) + 3  # a padded batch
        return st
    if op == "append":
        st["cache"] = torch.zeros(c["pages"], c["h"], 2, _page_bytes(c["page"], c["d"]),
                                  dtype=torch.uint8, device=DEV)
        # keys and values as a projection leaves them: slices of one row per token
        both = normal(c["t"], 2, c["h"], c["d"])
        st["k"], st["v"] = both[:, 0], both[:, 1]
        st["slots"] = torch.randperm(c["pages"] * c["page"], device=DEV, generator=g)[:c["t"]].int()
        return st
    b, page = c["b"], c["page"]
    width = -(-c["maxlen"] // page)
    lens = ints(c["minlen"], c["maxlen"] + 1, b)
    qlen = torch.randint(1, c["q"] + 1, (b,), generator=host, dtype=torch.int32).to(DEV)
    if c["ragged_q"]:
        qlen[0] = c["q"]
    else:
        qlen[:] = c["q"]
    st["lens"] = lens
    st["q_offsets"] = torch.cat([torch.zeros_like(qlen[:1]), qlen.cumsum(0).int()])
    st["q"] = normal(int(qlen.sum()), c["hq"], c["d"]) * 2
    st["table"] = torch.randperm(b * width, device=DEV, generator=g).int().view(b, width)
    st["cache"] = torch.empty(b * width, c["hk"], 2, _page_bytes(page, c["d"]), dtype=torch.uint8,
                              device=DEV)
    _fill_cache(st["cache"], page, c["d"], g)
    st["scale"] = 1.0 / math.sqrt(c["d"])
    return st


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _quantise(x):
    """Codes (two to a byte, the even one low) and e4m3 scale bytes of fp32 x[..., d]."""
    g = x.unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    t = torch.where(sf > 0, g / sf, torch.zeros_like(g))
    a = t.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)) | (torch.signbit(t).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _values(codes, scales):
    """fp32 values that code and scale bytes stand for."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    grid = torch.cat([grid, -grid])
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (grid[code].unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _parts(cache, page, d):
    return (cache[..., :page * d // 2].unflatten(-1, (page, d // 2)),
            cache[..., page * d // 2:].unflatten(-1, (page, d // GROUP)))


def _plain_rope(x, st):
    c = st["case"]
    r = c["r"]
    angle = st["positions"].double()[:, None] * st["freq"]
    angle = -angle if c["inverse"] else angle
    cos, sin = ((f(angle) * st["mscale"]).float() for f in (torch.cos, torch.sin))
    if c["layout"] == "tokens":
        cos, sin = cos[:, None], sin[:, None]
    xf = x.float()
    a, b = (xf[..., 0:r:2], xf[..., 1:r:2]) if c["interleaved"] else (xf[..., :r // 2], xf[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([y, z], -1).flatten(-2) if c["interleaved"] else torch.cat([y, z], -1)
    return torch.cat([y, xf[..., r:]], -1).to(x.dtype)


def _plain_plan(st):
    page = st["case"]["page"]
    lens, new, table, queue = st["lens"].long(), st["new"].long(), st["table"], st["queue"]
    b, width = table.shape
    cap = queue.numel()
    head, count = st["queue_state"][0].long(), st["queue_state"][1].long()
    done, add = new < 0, new.clamp(min=0)
    have, want = -(-lens // page), -(-(lens + add) // page)
    fits = want <= width
    need = torch.where(fits, want - have, 0)
    ok = fits & ((need == 0) | (need.cumsum(0) <= count))
    need = torch.where(ok, need, 0)
    back = torch.where(done, have, 0)
    i = torch.arange(width, device=DEV)[None]
    place = (need.cumsum(0) - need)[:, None] + i - have[:, None]
    taken = queue[(head + place) % cap]
    fresh = (i >= have[:, None]) & (i < (have + need)[:, None])
    # finished requests' pages go behind the free ones; everything else writes to a spare place
    at = (head + count + (back.cumsum(0) - back)[:, None] + i) % cap
    at = torch.where(i < back[:, None], at, cap)
    spare = torch.cat([queue, queue[:1]])
    spare[at.reshape(-1)] = table.reshape(-1)
    queue.copy_(spare[:-1])
    table.copy_(torch.where(fresh, taken, table))
    offsets = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0)])
    t = torch.arange(st["tokens"], device=DEV)
    r = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    real = r < b
    r = r.clamp(max=b - 1)
    pos = torch.where(real, lens[r] + t - offsets[r], 0)
    slot = table[r, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    slot = torch.where(real & ok[r], slot, -1)
    length = torch.where(done, 0, torch.where(ok, lens + add, lens))
    state = torch.stack([(head + need.sum()) % cap, count - need.sum() + back.sum()])
    return [length.int(), offsets.int(), pos.int(), slot.int(), state.int(), table, queue]


def _plain_append(st):
    c = st["case"]
    page, slots = c["page"], st["slots"].long()
    codes, scales = _parts(st["cache"], page, c["d"])
    p, i = slots // page, slots % page
    for n, x in enumerate((st["k"], st["v"])):
        q, s = _quantise(x.float())
        codes[p, :, n, i], scales[p, :, n, i] = q, s
    return [_values(codes[p, :, n, i], scales[p, :, n, i]).bfloat16() for n in (0, 1)]


def _plain_attend(st):
    c = st["case"]
    page, hk, d = c["page"], c["hk"], c["d"]
    b, width = st["table"].shape
    codes, scales = _parts(st["cache"], page, d)
    rows = st["table"].long()
    # [b, width, hk, 2, page, d] -> [2, b, hk, keys, d]
    kv = _values(codes[rows], scales[rows]).permute(3, 0, 2, 1, 4, 5).flatten(3, 4)
    lens, off = st["lens"].long(), st["q_offsets"].long()
    qlen = off[1:] - off[:-1]
    t = torch.arange(st["q"].shape[0], device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[r]
    q = torch.zeros(b, c["q"], c["hq"], d, device=DEV)
    q[r, i] = st["q"].float()
    q = q.permute(0, 2, 1, 3).reshape(b, hk, -1, d)  # heads of one key head side by side
    s = (q @ kv[0].transpose(-1, -2)) * st["scale"]
    j = torch.arange(width * page, device=DEV)
    last = lens[:, None] - 1
    if c["causal"]:
        last = last - qlen[:, None] + 1 + torch.arange(c["q"], device=DEV)[None]
    seen = (j <= last[..., None]) & (j < lens[:, None, None])  # [b, q or 1, keys]
    s = s.unflatten(2, (-1, c["q"]))
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ kv[1]).unflatten(2, (-1, c["q"])) / total.clamp(min=1e-38)
    lse = (m + torch.log(total)).squeeze(-1)
    o, lse = o.flatten(1, 2).transpose(1, 2), lse.flatten(1, 2).transpose(1, 2)
    return [o[r, i].to(torch.bfloat16), lse[r, i]]


def run(st):
    c, op = st["case"], st["op"]
    if own:
        import exact_attention_13_gb300 as ea

        if op == "rope":
            return ea.rope(st["q"], st["k"], st["positions"], st["turns"],
                           interleaved=c["interleaved"], inverse=c["inverse"], mscale=st["mscale"])
        if op == "plan":
            p = ea.page_plan(st["lens"], st["new"], st["table"], st["queue"], st["queue_state"],
                             page_size=c["page"], num_tokens=st["tokens"])
            return [p.lens, p.q_offsets, p.positions, p.slots, p.queue_state, st["table"], st["queue"]]
        if op == "append":
            ea.kv4_append(st["k"], st["v"], st["cache"], st["slots"])
            return ea.kv4_read(st["cache"], st["slots"], c["d"])
        return ea.kv4_fwd(st["q"], st["cache"], st["table"], st["lens"],
                          q_offsets=st["q_offsets"], max_q=c["q"], causal=c["causal"],
                          scale=st["scale"])
    if op == "rope":
        return (_plain_rope(st["q"], st), _plain_rope(st["k"], st))
    if op == "plan":
        return _plain_plan(st)
    if op == "append":
        return _plain_append(st)
    return _plain_attend(st)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op == "rope":
        n = c["b"] * c["n"] * (c["hq"] + c["hk"])
        return {"bytes": n * c["d"] * 4 + 4 * c["n"] + 4 * c["r"], "flops": 3 * n * c["r"]}
    if op == "plan":
        width = -(-c["maxlen"] // c["page"])
        mean = 1 if c["chunk"] == 1 else 0.6 + 0.3 * c["chunk"] / 2
        tokens = c["b"] * mean
        # lengths in and out, offsets, positions and slots; table entries that are added or freed
        moved = c["b"] * (mean / c["page"] + (0.05 * width / 2 if c["chunk"] > 1 else 0)) * 8
        return {"bytes": c["b"] * 16 + tokens * 8 + moved, "flops": 0}
    if op == "append":
        n = 2 * c["t"] * c["h"]
        # values read, cache bytes written, then read, values written
        return {"bytes": n * c["d"] * 4 + 2 * n * (c["d"] // 2 + c["d"] // GROUP) + 8 * c["t"],
                "flops": 4 * n * c["d"]}
    keys = c["b"] * (c["minlen"] + c["maxlen"]) / 2
    q = (c["q"] + 1) / 2 if c["ragged_q"] else c["q"]
    cache = keys * c["hk"] * 2 * (c["d"] // 2 + c["d"] // GROUP)
    seen = keys - (c["b"] * (q - 1) / 2 if c["causal"] else 0)
    return {"bytes": cache + c["b"] * q * c["hq"] * (4 * c["d"] + 4),
            "flops": 4 * c["d"] * c["hq"] * q * max(seen, c["b"])}


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


def _nearest(x, grid):
    """x >= 0 to the nearest of a sorted grid; a tie goes to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    down = (below < above) | ((below == above) & (hi % 2 == 1))
    return grid[torch.where(down, hi - 1, hi)]


def _exact_quantised(x):
    x = x.double().unflatten(-1, (-1, GROUP))
    n = torch.arange(127, device=x.device)
    e4m3 = torch.where(n < 8, (n % 8) * 2.0 ** -9, (1 + (n % 8) / 8) * 2.0 ** ((n // 8).double() - 7)).double()
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    s = _nearest(x.abs().amax(-1) / 6, e4m3)[..., None]
    return (torch.sign(x) * _nearest(torch.where(s > 0, x.abs() / s, 0.0), e2m1) * s).flatten(-2)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "plan":
        return None  # whole numbers only
    if c["op"] == "append":
        return [_exact_quantised(st["k"]), _exact_quantised(st["v"])]
    if c["op"] == "rope":
        out = []
        turn = torch.exp(1j * st["positions"].double()[:, None] * st["freq"]) * st["mscale"]
        turn = turn.conj() if c["inverse"] else turn
        turn = turn[:, None] if c["layout"] == "tokens" else turn
        for x in (st["q"], st["k"]):
            y = x.double()
            h = c["r"] // 2
            first = slice(0, c["r"], 2) if c["interleaved"] else slice(0, h)
            second = slice(1, c["r"], 2) if c["interleaved"] else slice(h, c["r"])
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            out.append(y)
        return tuple(out)
    page, d, group = c["page"], c["d"], c["hq"] // c["hk"]
    off = st["q_offsets"].tolist()
    outs, lses = [], []
    for b, n in enumerate(st["lens"].tolist()):
        blocks = st["cache"][st["table"][b, :-(-n // page)].long()]  # [pages, hk, 2, bytes]
        codes = blocks[..., :page * d // 2].reshape(*blocks.shape[:3], page, -1)
        scales = blocks[..., page * d // 2:].reshape(*blocks.shape[:3], page, -1)
        kv = _decode(codes, scales).permute(2, 1, 0, 3, 4).reshape(2, c["hk"], -1, d)[:, :, :n]
        q = st["q"][off[b]:off[b + 1]].double().transpose(0, 1)  # [hq, rows, d]
        rows = q.shape[1]
        o, lse = torch.empty_like(q), torch.empty_like(q[..., 0])
        for h in range(c["hq"]):
            x = st["scale"] * q[h] @ kv[0, h // group].T
            if c["causal"]:
                above = torch.ones(rows, n, dtype=torch.bool, device=x.device).triu(n - rows + 1)
                x = x.masked_fill(above, -math.inf)
            lse[h] = torch.logsumexp(x, -1)
            o[h] = torch.exp(x - lse[h][:, None].clamp(min=-1e300)) @ kv[1, h // group]
        outs.append(o.transpose(0, 1))
        lses.append(lse.transpose(0, 1))
    return [torch.cat(outs), torch.cat(lses)]
