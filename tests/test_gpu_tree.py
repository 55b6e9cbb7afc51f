"""Trees of drafted tokens over the 4-bit cache on the GPU against the fp64 reference: plan, acceptance and moves
(integers and bytes: equal), and attention."""
import math

import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import tree

pytestmark = pytest.mark.gpu


def numpy64(t):
    return t.double().cpu().numpy()


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def offsets_of(nodes):
    return np.concatenate([[0], np.cumsum(nodes)]).tolist()


def random_trees(rng, nodes, spread=6, wild=False):
    """Parents, packed; node 0 hangs on the cached token, `wild`: so do some others, and some parents are none."""
    out = []
    for n in nodes:
        p = [-1] + [i - 1 - int(rng.integers(0, min(i, spread))) for i in range(1, n)]
        if wild:
            for i in range(n):
                if rng.random() < 0.2:
                    p[i] = int(rng.choice([-1, -7, i, i + 3, 2 ** 31 - 1, -2 ** 31]))
        out += p[:n]
    return out


# --------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("nodes,max_nodes,spread", [
    ([1], 1, 1), ([9, 0, 5, 1, 32, 33], 33, 4), ([64] * 5, 64, 1), ([256, 255, 129, 1, 0, 200], 256, 1),
    ([256, 100], 256, 300), ([7] * 700, 7, 3), ([300, 40, 270, 1000], 256, 1), ([50, 3], 20, 5), ([0, 0, 0], 8, 1),
    ([700, 2, 1700], 40, 1), ([900, 129, 33], 1, 200), ([1500], 256, 400),
])
@pytest.mark.parametrize("wild", [False, True])
def test_plan(nodes, max_nodes, spread, wild):
    rng = np.random.default_rng(len(nodes) + max_nodes)
    parents, off = random_trees(rng, nodes, spread, wild), offsets_of(nodes)
    lens = rng.integers(0, 5000, len(nodes)).tolist()
    words = -(-max_nodes // 32)
    for T in {off[-1] + 3, off[-1], max(1, off[-1] - 2)}:  # padded, whole, cut short
        p = (parents + [0] * 3)[:T]
        if not p:
            continue
        want = tree.tree_plan(p, off, lens, words)
        got = ea.tree_plan(ints(p), ints(off), ints(lens), max_nodes)
        assert got.positions.tolist() == want[0].tolist()
        assert np.array_equal(got.seen.cpu().numpy(), tree.bits(want[1]))


def test_plan_bad_offsets_and_refusals():
    """Offsets outside the rows, or falling, stay inside the buffers; rows of no request are not looked at."""
    p, lens = ints([-1, 0, 1, 2]), ints([5, 6])
    for off in ([0, -3, 900], [2, 1, 4], [-5, 2, 4], [2 ** 31 - 1, 0, 2]):
        ea.tree_plan(p, ints(off), lens, 4)
    torch.cuda.synchronize()
    off = ints([0, 2, 4])
    out = ea.tree_plan(p, off, lens, 40)
    again = ea.tree_plan(p, off, lens, 40, out=out)
    assert again.seen.shape == (4, 2) and again.positions.tolist() == [5, 6, 6, 6]
    for bad in (dict(parents=p.long()), dict(q_offsets=off[:2]), dict(max_nodes=0), dict(max_nodes=257),
                dict(lens=lens.cpu()), dict(out=ea.TreePlan(out[0], out[1][:, :1])), dict(parents=p[::2])):
        with pytest.raises(ValueError):
            ea.tree_plan(**(dict(parents=p, q_offsets=off, lens=lens, max_nodes=40) | bad))
    assert ea.tree_plan(p[:0], ints([0, 0, 0]), lens, 4).positions.shape == (0,)


@pytest.mark.parametrize("max_nodes,room", [(1, 32), (5, 32), (20, 32), (32, 32), (33, 64), (250, 256)])
def test_max_nodes_counts_whole_words(max_nodes, room):
    """A chain longer than `max_nodes`: nodes up to the next multiple of 32 have bits and can be accepted, no others."""
    n = room + 9
    parents, off, lens = ints(range(-1, n - 1)), ints([0, n]), ints([7])
    got = ea.tree_plan(parents, off, lens, max_nodes)
    assert got.seen.shape == (n, room // 32) and got.positions.tolist() == list(range(7, 7 + n))
    whole = ea.tree_plan(parents, off, lens, room)
    assert torch.equal(got.seen, whole.seen)
    bits = (got.seen.cpu().numpy().view(np.uint32)[:, :, None] >> np.arange(32, dtype=np.uint32) & 1).reshape(n, -1)
    assert np.array_equal(bits, np.tril(np.ones((n, n), dtype=int))[:, :room])
    one = ints([1] * n)
    step = ea.tree_accept(parents, got.seen, one, one, lens, ints([7 + n]), off, ints(range(7, 7 + n)),
                          ints(np.zeros((1, 30))), ints([0] * 30), ints([0, 0]), 16)
    assert step.counts.tolist() == [room] and step.lens.tolist() == [7 + room]


# --------------------------------------------------------------------------------- acceptance
def accept_case(rng, nodes, page, wild=False, refuse=0.1, end=0.1, vocabulary=3):
    B, off = len(nodes), offsets_of(nodes)
    lens = rng.integers(0, 200, B)
    new = lens + np.asarray(nodes)
    width = int(-(-(200 + max(nodes)) // page))
    table = rng.permutation(B * width).reshape(B, width)
    slots = []
    for b, n in enumerate(nodes):
        kind = rng.random()
        if kind < refuse:
            new[b] = lens[b]
        slots += [int(table[b, j // page]) * page + j % page if new[b] > lens[b] else -1
                  for j in range(lens[b], lens[b] + n)]
        if n == 0 and kind > 1 - end:
            new[b] = 0
    have = -(-new // page)
    spare = np.concatenate([table[b, have[b]:] for b in range(B)])
    cap = B * width
    queue = np.full(cap, -7)
    head = 3 % cap
    queue[(head + np.arange(len(spare))) % cap] = spare
    T = off[-1]
    return dict(parents=random_trees(rng, nodes, 5, wild), tokens=rng.integers(0, vocabulary, T).tolist(),
                choices=rng.integers(0, vocabulary, T).tolist(), lens=lens.tolist(), new_lens=new.tolist(),
                q_offsets=off, slots=slots, table=table.tolist(), queue=queue.tolist(), queue_state=[head, len(spare)])


def run_accept(c, page, words, T=None, seen=None):
    T = len(c["parents"]) if T is None else T
    cut = {k: (c[k] + [0] * T)[:T] for k in ("parents", "tokens", "choices", "slots")}
    c = c | cut
    if seen is None:
        seen = tree.bits(tree.tree_plan(c["parents"], c["q_offsets"], c["lens"], words)[1])
    queue = ints(c["queue"])
    got = ea.tree_accept(ints(c["parents"]), ints(seen).view(T, words), ints(c["tokens"]), ints(c["choices"]),
                         ints(c["lens"]), ints(c["new_lens"]), ints(c["q_offsets"]), ints(c["slots"]), ints(c["table"]),
                         queue, ints(c["queue_state"]), page)
    return [*(t.tolist() for t in got), queue.tolist()], c


@pytest.mark.parametrize("nodes,page,words", [
    ([1], 16, 1), ([9] * 8, 64, 1), ([12, 0, 1, 33, 5, 0, 64, 2], 16, 2), ([256, 128, 129, 1, 255], 128, 8),
    ([20] * 600, 32, 1), ([300, 9, 270], 16, 8), ([40, 50], 32, 1), ([0, 0, 3], 16, 1), ([2] * 16384, 16, 1),
    ([5, 1, 0] * 3, 16, 1), ([70, 3, 9, 0] * 9 + [256], 32, 8), ([6, 3] * 32, 16, 1), ([6] * 65, 16, 1),
])
@pytest.mark.parametrize("wild", [False, True])
def test_accept(nodes, page, words, wild):
    rng = np.random.default_rng(sum(nodes) + page)
    c = accept_case(rng, nodes, page, wild)
    names = ("lens", "counts", "path", "next_tokens", "sources", "queue_state", "queue")
    for T in {len(c["parents"]), len(c["parents"]) + 3, max(1, len(c["parents"]) - 4)}:
        got, d = run_accept(c, page, words, T)
        want = tree.tree_accept(d["parents"], d["tokens"], d["choices"], d["lens"], d["new_lens"], d["q_offsets"],
                                d["slots"], d["table"], d["queue"], d["queue_state"], page, words)
        for name, g, w in zip(names, got, want):
            assert g == [int(x) for x in w], name


def test_accept_without_nodes_a_full_ring_and_meaningless_bits():
    rng = np.random.default_rng(7)
    c = accept_case(rng, [5, 8, 3], 16, refuse=0.0)
    c["new_lens"] = [n + 40 for n in c["new_lens"]]  # pages for more tokens than the nodes: they all come back
    c["queue"], c["queue_state"] = [-7] * 5, [4, 3]  # and do not fit
    got, d = run_accept(c, 16, 1)
    want = tree.tree_accept(d["parents"], d["tokens"], d["choices"], d["lens"], d["new_lens"], d["q_offsets"],
                            d["slots"], d["table"], d["queue"], d["queue_state"], 16, 1)
    assert got == [[int(x) for x in w] for w in want] and got[5] == [4, 5]
    # bits that belong to no tree of these parents: any answer inside the buffers
    for word in (0, -1, -2 ** 31, 0x55555555):
        got, _ = run_accept(c, 16, 1, seen=np.full((16, 1), word))
        assert all(0 <= n <= 8 for n in got[1]) and all(-1 <= p < 8 for p in got[2])
    none = ints([])
    got = ea.tree_accept(none, none.view(0, 1), none, none, ints([7, 9]), ints([0, 9]), ints([0, 0, 0]), none,
                         ints([[1], [2]]), ints([5, 6]), ints([0, 1]), 16)
    assert [t.tolist() for t in got] == [[0, 9], [0, 0], [], [-1, -1], [], [0, 1]]


def test_accept_refusals():
    c = accept_case(np.random.default_rng(1), [3, 4], 16)
    args = {k: ints(c[k]) for k in ("parents", "tokens", "choices", "lens", "new_lens", "q_offsets", "slots", "table",
                                    "queue", "queue_state")}
    args |= dict(seen=ints([[1]] * 7), page_size=16)
    out = ea.tree_accept(**args)
    for bad in (dict(tokens=args["tokens"][:3]), dict(choices=args["choices"].long()), dict(seen=ints([[0] * 9] * 7)),
                dict(seen=args["seen"][:, 0]), dict(slots=args["slots"].cpu()), dict(queue_state=ints([1, 2, 3])),
                dict(table=args["table"][:1]), dict(page_size=0), dict(out=out._replace(path=out.path[:2]))):
        with pytest.raises(ValueError):
            ea.tree_accept(**(args | bad))
    for bad in (dict(page_size=24), dict(out=out._replace(lens=args["lens"])),
                dict(out=out._replace(queue_state=args["queue_state"]))):
        with pytest.raises(ea.AttentionError):
            ea.tree_accept(**(args | bad))


# --------------------------------------------------------------------------------- moves
@pytest.mark.parametrize("d,page,H,layers", [(128, 16, 1, 1), (64, 32, 3, 5), (128, 64, 8, 2), (64, 128, 2, 256)])
def test_move(d, page, H, layers):
    rng = np.random.default_rng(layers)
    pages, counts, lens = 12, [3, 0, 9, 20, 1], [6, 4, 12, 30, 2]
    off = offsets_of(lens)
    place = rng.permutation(pages * page)[:off[-1]]
    slots, sources = place.copy(), np.full(off[-1], -1)
    for b, n in enumerate(lens):  # rising nodes of each request, at or behind their places
        path = np.sort(rng.permutation(n)[:counts[b]])
        sources[off[b]:off[b] + counts[b]] = place[off[b] + path]
    sources[off[3] + 2], slots[off[3] + 5] = pages * page, -1  # rows that go nowhere or come from nowhere
    cache = torch.randint(0, 256, (layers, pages, H, 2, page * 9 * d // 16), dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(1)).cuda()
    want = [tree.kv4_move(x, sources, slots, off, counts, d) for x in cache.cpu().numpy()]
    apart = [x.clone() for x in cache]
    args = (ints(sources), ints(slots), ints(off), ints(counts), d)
    ea.kv4_move(apart, *args)
    if layers == 1:
        one = cache[0].clone()
        ea.kv4_move(one, *args)
        assert np.array_equal(one.cpu().numpy(), want[0])
    ea.kv4_move(cache, *args)
    for x, y, w in zip(cache, apart, want):
        assert np.array_equal(x.cpu().numpy(), w) and torch.equal(x, y)


def test_move_refusals_and_counts():
    cache = ea.kv4_cache(4, 2, 16, 64)
    i = ints([0, 1, 2, 3])
    off, counts = ints([0, 4]), ints([2])
    for bad in (([cache, cache], i, i, off, counts, 64), ([cache, ea.kv4_cache(5, 2, 16, 64)], i, i, off, counts, 64),
                (cache, i, i[:3], off, counts, 64), (cache, i, i, off[:1], counts, 64), (cache, i, i, off, counts, 128),
                (cache, i.cpu(), i, off, counts, 64), (torch.stack([cache] * 257), i, i, off, counts, 64),
                (cache[None].expand(3, -1, -1, -1, -1), i, i, off, counts, 64)):
        with pytest.raises(ValueError):
            ea.kv4_move(*bad)
    # counts past the rows of a request, and negative ones, move what there is
    cache.random_(0, 256)
    want = cache.clone()
    ea.kv4_move(want, ints([40, 41, 42, 43]), i, off, ints([4]), 64)
    got = cache.clone()
    ea.kv4_move(got, ints([40, 41, 42, 43]), i, off, ints([2 ** 31 - 1]), 64)
    assert torch.equal(got, want) and not torch.equal(got, cache)
    got = cache.clone()
    ea.kv4_move(got, ints([40, 41, 42, 43]), i, off, ints([-1]), 64)
    assert torch.equal(got, cache)
    ea.kv4_move(got, i[:0], i[:0], ints([0, 0]), ints([0]), 64)


# --------------------------------------------------------------------------------- attention
def make(lens, width, page, Hkv, d, seed=0, extra=3):
    """A cache of normal keys and values with scattered pages, and its table.  Bytes that no request
    owns are 0xff: NaN scales."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    pages = B * width + extra
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    cache = torch.full((pages, Hkv, 2, page * 9 * d // 16), 255, dtype=torch.uint8).cuda()
    slots = []
    for b, m in enumerate(lens):
        j = np.arange(max(0, min(m, width * page)))
        slots += (table[b, j // page] * page + j % page).tolist()
    if slots:
        k, v = normal(len(slots), Hkv, d, seed=seed + 1), normal(len(slots), Hkv, d, seed=seed + 2)
        k[:, :, 3] *= 6
        ea.kv4_append(k.bfloat16().cuda(), v.bfloat16().cuda(), cache, ints(slots))
    return cache, table


def queries(T, Hq, d, seed=9):
    return (normal(T, Hq, d, seed=seed) * 2).bfloat16().cuda()


def check(q, cache, table, lens, offsets, seen, d, scale=None, kd=1.0, vd=1.0, got=None, **kw):
    """Tolerances.  A score is a sum of exact products in fp32 (d roundings at most, some by truncation) of
    queries rounded 2^-25 of the row's largest value: off by delta = 2^-18 scale sum|q k| at most.  p then is off
    by delta relative, f16 P by 2^-11 relative or, where it is subnormal, half of 2^-24 absolute with the row's
    largest P at 2^7 or more (2^-32 of it: sum p is at least the largest, so O is off by 2^-32 sum |v|), ex2 by
    2^-21, and O = sum p v / sum p by the relative part twice over; bf16 O by 2^-8.  LSE is off by delta and fp32
    roundings of a few 2^-22 (1 + |LSE|)."""
    scale = 1 / math.sqrt(d) if scale is None else scale
    o64, lse64, mass, total, dot = tree.kv4_tree_attention(numpy64(q), cache.cpu().numpy(), np.asarray(table), lens,
                                                           offsets, seen, d, scale, kd, vd)
    if got is None:
        got = ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(offsets), ints(tree.bits(seen)), scale=scale,
                              k_descale=kd, v_descale=vd, **kw)
    o, lse = (numpy64(t) for t in got)
    n = min(offsets[-1], len(o))
    o64, lse64, mass, total = o64[:n], lse64[:n], mass[:n], total[:n]
    delta = 2.0 ** -18 * scale * dot[:n]
    tol = 2.0 ** -8 * np.abs(o64) + (2 * delta[..., None] + 2.0 ** -10) * mass + 2.0 ** -32 * total
    finite = np.isfinite(lse64)
    assert (np.abs(o[:n] - o64) <= tol).all(), np.nanmax(np.abs(o[:n] - o64) / tol)
    assert np.array_equal(np.isneginf(lse[:n]), ~finite)
    err = np.abs(lse[:n] - np.where(finite, lse64, 0))[finite]
    lim = (delta + 2.0 ** -20 * (1 + np.abs(np.where(finite, lse64, 0))))[finite]
    assert (err <= lim).all(), (err / lim).max()
    return got


def trees_of(nodes, seed=0, words=None, T=None):
    rng = np.random.default_rng(seed)
    words = words or -(-max(max(nodes), 1) // 32)
    parents = random_trees(rng, nodes)
    T = len(parents) if T is None else T
    return tree.tree_plan((parents + [0] * T)[:T], offsets_of(nodes), [0] * len(nodes), words)[1]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (7, 1), (24, 2)])
def test_lengths(d, page, Hq, Hkv):
    lens = [1, 0, 15, 16, 17, 31, 33, 127, 128, 129, 300, 500]
    nodes = [1, 2, 9, 16, 5, 1, 3, 8, 12, 7, 4, 10]
    cache, table = make(lens, -(-500 // page), page, Hkv, d)
    check(queries(sum(nodes), Hq, d), cache, table, lens, offsets_of(nodes), trees_of(nodes), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,nodes", [
    (4, 1, [2, 0, 1, 3, 4]), (4, 4, [9, 1, 7, 8, 16]), (6, 2, [11, 5, 12, 0, 6]), (1, 1, [31, 32, 33, 1, 17]),
    (3, 1, [43, 3, 20, 1, 42]), (16, 2, [130, 2, 33, 5, 1]), (2, 1, [256, 64, 65, 128, 255]),
])
def test_blocks_of_rows(d, Hq, Hkv, nodes):
    """Blocks of all sizes, several of them, trees longer than the cache, requests without keys or nodes."""
    lens = [130, 64, 5, 0, 333]
    cache, table = make(lens, 6, 64, Hkv, d)
    seen, off = trees_of(nodes), offsets_of(nodes)
    q = queries(off[-1], Hq, d)
    for max_q in (max(nodes), 1, 5, 300):
        check(q, cache, table, lens, off, seen, d, max_q=max_q)


@pytest.mark.parametrize("rows", [8, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_any_mask_of_bits(rows, d):
    """Masks that are no trees, and rows whose mask leaves nothing in a request that is all tree."""
    rng = np.random.default_rng(rows)
    nodes, lens = [rows, rows, rows], [rows, rows + 130, max(0, rows - 3)]
    cache, table = make(lens, 11, 32, 2, d)
    seen = rng.random((3 * rows, 32 * -(-rows // 32))) < 0.3
    seen[::3] = False
    got = check(queries(3 * rows, 2, d), cache, table, lens, offsets_of(nodes), seen, d, max_q=rows)
    assert bool(torch.isneginf(got[1]).any()) and bool((got[0][0] == 0).all())


@pytest.mark.parametrize("d,page,lens,nodes,Hq,Hkv", [
    (128, 64, [20000], [5], 8, 1), (64, 16, [9000, 3], [20, 3], 4, 1), (128, 128, [5000, 0, 7001, 1], [30, 1, 33, 1], 4, 2),
    (128, 32, [30000], [64], 2, 1), (64, 64, [25000, 400], [3, 1], 8, 4), (128, 16, [9000, 800], [100, 255], 2, 2),
])
def test_long_caches_split_over_the_gpu(d, page, lens, nodes, Hq, Hkv):
    cache, table = make(lens, -(-max(lens) // page), page, Hkv, d)
    off, seen = offsets_of(nodes), trees_of(nodes)
    q = queries(off[-1], Hq, d)
    size = ea.kv4_tree_workspace_bytes(Hq, Hkv, d, max(nodes), page, table.shape[1])
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    a = check(q, cache, table, lens, off, seen, d, max_q=max(nodes), workspace=ws)
    b = ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), ints(tree.bits(seen)), max_q=max(nodes),
                        workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits again


def test_many_short_requests():
    rng = np.random.default_rng(4)
    lens, nodes = rng.integers(0, 70, 700).tolist(), rng.integers(0, 6, 700).tolist()
    cache, table = make(lens, 5, 16, 1, 64)
    check(queries(sum(nodes), 2, 64), cache, table, lens, offsets_of(nodes), trees_of(nodes), 64, max_q=5)


def on_gpu(q, cache, table, lens, offsets, seen, d):
    """The attention of the 64-bit reference, one request and key head at a time on the GPU, with the tolerances' sums
    of |q k|, of p |v| and of |v|."""
    T, Hq, _ = q.shape
    Hkv, page = cache.shape[1], cache.shape[3] * 16 // (9 * d)
    o, lse = torch.zeros(T, Hq, d).double().cuda(), torch.full((T, Hq), -math.inf).double().cuda()
    mass, total, dot = torch.zeros_like(o), torch.zeros_like(o), torch.zeros_like(lse)
    G = Hq // Hkv
    for b, n in enumerate(lens):
        at, m = torch.arange(n).cuda(), offsets[b + 1] - offsets[b]
        if n == 0 or m == 0:
            continue
        slots = (torch.as_tensor(table[b]).cuda()[at // page] * page + at % page).int()
        k, v = (x.double() for x in ea.kv4_read(cache, slots, d))
        rows = slice(offsets[b], offsets[b + 1])
        live = torch.ones(m, n, dtype=torch.bool, device="cuda")
        w = min(m, n)  # nodes that are cached: the last ones of the tree fill the cache
        live[:, n - m if n >= m else 0:] = torch.as_tensor(seen[rows, max(0, m - n):m]).cuda()[:, :w]
        for h in range(Hkv):
            x = q[rows, h * G:(h + 1) * G].double()
            s = torch.einsum("mgd,nd->mgn", x, k[:, h]) / math.sqrt(d)
            s = s.masked_fill(~live[:, None], -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.where(torch.isfinite(s), torch.exp(s - torch.where(torch.isfinite(top), top, 0)), 0)
            sum_ = p.sum(-1, keepdim=True)
            some = sum_ > 0
            p = torch.where(some, p / torch.where(some, sum_, 1), 0)
            cols = slice(h * G, (h + 1) * G)
            lse[rows, cols] = torch.where(some, top + torch.log(sum_), -math.inf)[..., 0]
            o[rows, cols] = torch.einsum("mgn,nd->mgd", p, v[:, h])
            mass[rows, cols] = torch.einsum("mgn,nd->mgd", p, v[:, h].abs())
            total[rows, cols] = v[:, h].abs().sum(0)
            dot[rows, cols] = torch.einsum("mgd,nd->mgn", x.abs(), k[:, h].abs()).amax(-1)
    return o, lse, mass, total, dot


@pytest.mark.parametrize("d,Hq,Hkv,most,nodes", [
    (128, 16, 4, 8000, 16), (64, 16, 8, 9000, 16), (128, 32, 8, 7000, 7), (128, 8, 4, 8000, 60), (64, 12, 4, 9000, 50),
    (128, 8, 8, 6000, 3), (128, 16, 8, 6000, 8),
])
def test_many_tiles_a_share(d, Hq, Hkv, most, nodes):
    """Ragged requests, some short ones among them, with enough tiles that the shares count what units cost."""
    rng = np.random.default_rng(nodes)
    long = -(-2800 * 128 // (Hkv * most * 3 // 4))
    lens = [n + nodes for n in rng.integers(most // 2, most, long).tolist() + rng.integers(0, 300, 10).tolist()]
    lens = [lens[i] for i in rng.permutation(len(lens))] + [0, 1]
    trees = rng.integers(1, nodes + 1, len(lens)).tolist()
    tiles = sum(-(-n // 128) for n in lens) * Hkv
    assert tiles > 16 * 152 or max(trees) * Hq // Hkv <= 16
    cache, table = make(lens, -(-max(lens) // 64), 64, Hkv, d)
    off, seen = offsets_of(trees), trees_of(trees)
    q = queries(off[-1], Hq, d)
    o64, lse64, mass, total, dot = on_gpu(q, cache, table, lens, off, seen, d)
    ws = torch.full((ea.kv4_tree_workspace_bytes(Hq, Hkv, d, nodes, 64, table.shape[1]),), 255, dtype=torch.uint8).cuda()
    o, lse = ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), ints(tree.bits(seen)), max_q=nodes,
                             workspace=ws)
    delta = 2.0 ** -18 * dot / math.sqrt(d)  # (as in `check`)
    tol = 2.0 ** -8 * o64.abs() + (2 * delta[..., None] + 2.0 ** -10) * mass + 2.0 ** -32 * total
    assert bool(((o.double() - o64).abs() <= tol).all())
    some = torch.isfinite(lse64)
    assert torch.equal(torch.isneginf(lse), ~some)
    assert bool(((lse.double() - lse64).abs() <= delta + 2.0 ** -20 * (1 + lse64.abs()))[some].all())


@pytest.mark.parametrize("max_q", [3, 8, 20])  # units of 32, 64 and 256 rows
def test_more_requests_than_threads_with_many_tiles(max_q):
    rng = np.random.default_rng(max_q)
    lens, nodes = rng.integers(0, 70, 1400).tolist(), rng.integers(0, 6, 1400).tolist()
    lens[700] = 900
    cache, table = make(lens, 57, 16, 2, 64)
    off, seen = offsets_of(nodes), trees_of(nodes)
    q = queries(off[-1], 16, 64)
    o64, lse64, mass, total, dot = on_gpu(q, cache, table, lens, off, seen, 64)
    o, lse = ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), ints(tree.bits(seen)), max_q=max_q)
    delta = 2.0 ** -18 * dot / math.sqrt(64)  # (as in `check`)
    tol = 2.0 ** -8 * o64.abs() + (2 * delta[..., None] + 2.0 ** -10) * mass + 2.0 ** -32 * total
    assert bool(((o.double() - o64).abs() <= tol).all())
    some = torch.isfinite(lse64)
    assert torch.equal(torch.isneginf(lse), ~some)
    assert bool(((lse.double() - lse64).abs() <= delta + 2.0 ** -20 * (1 + lse64.abs()))[some].all())


@pytest.mark.parametrize("max_q", [1, 12, 40, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_far_scores_rescale_the_sums(d, max_q):
    """Keys that grow along the cache: the maximum moves by hundreds of powers of two from tile to tile."""
    lens, nodes = [900, 130], [40, 9]
    cache, table = make(lens, 57, 16, 1, d)
    for b, n in enumerate(lens):
        j = np.arange(n)
        slots = table[b, j // 16] * 16 + j % 16
        k = (normal(n, 1, d, seed=b) * torch.linspace(0.1, 60, n)[:, None, None]).bfloat16().cuda()
        ea.kv4_append(k, normal(n, 1, d, seed=5).bfloat16().cuda(), cache, ints(slots))
    check(queries(49, 3, d), cache, table, lens, offsets_of(nodes), trees_of(nodes), d, max_q=max_q)
    down = queries(49, 3, d)
    down[::2] *= 1e-30
    down[1::4] *= 1e4
    check(down, cache, table, lens, offsets_of(nodes), trees_of(nodes), d, max_q=max_q, scale=0.5)


@pytest.mark.parametrize("max_q", [1, 5, 7, 12, 20, 40, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_all_magnitudes_share_a_pass(d, max_q):
    """A row keeps its bits whatever the others of its request hold: as small as 2^-120 of them, or zero."""
    lens, nodes = [300, 130], [40, 9]
    cache, table = make(lens, 19, 16, 1, d)
    off, seen = offsets_of(nodes), trees_of(nodes)
    for up in (1e4, 1e8, 1e20, 1e36):
        q = queries(49, 3, d).float()
        q[5::17] *= up
        q[3::11] = 0
        q[7::13, 1] *= 2.0 ** -15
        check(q.bfloat16(), cache, table, lens, off, seen, d, max_q=max_q, scale=0.5)


@pytest.mark.parametrize("max_q", [2, 20, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_not_a_number_reaches_the_rows_that_see_it(d, max_q):
    """NaN keys and values, in the tree and before it, and an infinite query."""
    lens, nodes = [200, 150, 64], [20, 9, 20]
    cache, table = make(lens, 7, 32, 1, d)
    seen, off = trees_of(nodes), offsets_of(nodes)
    q = queries(off[-1], 2, d)
    clean = check(q, cache, table, lens, off, seen, d, max_q=max_q)
    bad = torch.full((1, 1, d), math.nan).bfloat16().cuda()
    fine = normal(1, 1, d).bfloat16().cuda()
    slot = lambda b, j: ints([table[b, j // 32] * 32 + j % 32])  # noqa: E731
    ea.kv4_append(bad, fine, cache, slot(0, 200 - 20 + 7))   # node 7's key
    ea.kv4_append(fine, bad, cache, slot(0, 200 - 20 + 11))  # node 11's value
    ea.kv4_append(fine, bad, cache, slot(1, 3))              # a value before the tree: the whole request
    q[off[2] + 4, 1, 5] = math.inf
    o, lse = ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), ints(tree.bits(seen)), max_q=max_q)
    hit = torch.zeros(off[-1], 2, dtype=torch.bool)
    hit[:20] = torch.tensor(seen[:20, 7] | seen[:20, 11])[:, None]
    hit[20:29] = True
    hit[off[2] + 4, 1] = True
    hit = hit.cuda()
    assert bool(hit.any()) and not bool(hit.all())
    assert bool(torch.isnan(lse[hit]).all()) and bool(torch.isnan(o[hit]).all())
    same = ~hit
    same[:20] = False  # (node 11's new key and the finite rows of request 0 are checked by the reference below)
    assert torch.equal(o[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])
    assert bool(torch.isfinite(o[:20][~hit[:20]]).all()) and bool(torch.isfinite(lse[:20][~hit[:20]]).all())


@pytest.mark.parametrize("max_q", [1, 8, 16, 20, 64])  # units of 8, 16, 32, 64 and 256 rows
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_do_not_see_it_lie_within_the_reference(d, max_q):
    """Rows that share tiles with NaN keys and values of their own tree, and do not see them: the 64-bit reference of the
    cache without them, within the tolerances of `check`."""
    lens, nodes = [200, 150, 64], [20, 9, 20]
    cache, table = make(lens, 7, 32, 1, d)
    seen, off = trees_of(nodes), offsets_of(nodes)
    q = queries(off[-1], 2, d)
    o64, lse64, mass, total, dot = tree.kv4_tree_attention(numpy64(q), cache.cpu().numpy(), table, lens, off, seen, d,
                                                           1 / math.sqrt(d))
    bad = torch.full((1, 1, d), math.nan).bfloat16().cuda()
    fine = normal(1, 1, d, seed=3).bfloat16().cuda() * 8
    for b, node, key in ((0, 7, True), (0, 11, False), (2, 13, True)):
        j = lens[b] - nodes[b] + node
        ea.kv4_append(*((bad, fine) if key else (fine, bad)), cache, ints([table[b, j // 32] * 32 + j % 32]))
    o, lse = (numpy64(t) for t in ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), ints(tree.bits(seen)),
                                                  max_q=max_q))
    free = np.ones(off[-1], dtype=bool)
    free[:20] = ~(seen[:20, 7] | seen[:20, 11])
    free[off[2]:] = ~seen[off[2]:, 13]
    assert 3 <= free[:20].sum() < 20 and free[off[2]:].sum() < 20
    assert np.isnan(o[~free]).all() and np.isnan(lse[~free]).all()
    delta = 2.0 ** -18 / math.sqrt(d) * dot
    tol = 2.0 ** -8 * np.abs(o64) + (2 * delta[..., None] + 2.0 ** -10) * mass + 2.0 ** -32 * total
    assert (np.abs(o - o64) <= tol)[free].all()
    assert (np.abs(lse - lse64) <= delta + 2.0 ** -20 * (1 + np.abs(lse64)))[free].all()


@pytest.mark.parametrize("nodes", [3, 20, 50])
def test_missing_pages_bad_lengths_and_cut_batches(nodes):
    d, page = 128, 16
    lens, count = [300, 170, 90], [nodes, nodes, nodes]
    cache, table = make(lens, 19, page, 2, d)
    table = table.copy()
    table[0, 3], table[0, 18], table[1, 0], table[2, 5] = -1, 10 ** 6, len(cache), -2 ** 31
    off, seen = offsets_of(count), trees_of(count)
    q = queries(off[-1], 4, d)
    check(q, cache, table, lens, off, seen, d, max_q=nodes)
    # lengths past the table are clamped, as in the reference; negative ones leave no keys
    for bad in ([10 ** 6, 304, -4], [2 ** 31 - 1, -2 ** 31, 0]):
        cache2, table2 = make([304, 304, 304], 19, page, 2, d)
        check(q, cache2, table2, bad, off, seen, d, max_q=nodes)
    # a batch cut short: the rows that there are keep their places; rows behind the last request stay
    cut = off[-1] - nodes // 2
    check(q[:cut].contiguous(), cache, table, lens, off, seen[:cut], d, max_q=nodes)
    pad = torch.cat([q, queries(5, 4, d)])
    out = torch.full_like(pad, 7)
    lse = torch.full((off[-1] + 5, 4), 7.0).cuda()
    more = np.concatenate([seen, np.ones((5, seen.shape[1]), dtype=bool)])
    check(pad, cache, table, lens, off, more, d, max_q=nodes, out=out, lse=lse)
    assert bool((out[off[-1]:] == 7).all()) and bool((lse[off[-1]:] == 7).all())
    for odd in ([0, -3, 900, 2], [5, 1, 4, 9], [2 ** 31 - 1, 0, 2, 4]):  # offsets that make no sense: inside the buffers
        ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(odd), ints(tree.bits(seen)), max_q=nodes)
    torch.cuda.synchronize()


@pytest.mark.parametrize("nodes,words", [(70, 2), (40, 1), (300, 8)])
def test_nodes_past_the_bits_are_not_seen(nodes, words):
    lens, count = [400], [nodes]
    cache, table = make(lens, 7, 64, 1, 64)
    seen = np.random.default_rng(0).random((nodes, 32 * words)) < 0.5
    check(queries(nodes, 1, 64), cache, table, lens, offsets_of(count), seen, 64, max_q=nodes)


@pytest.mark.parametrize("nodes", [4, 16, 33])
def test_strides_streams_descales_and_captured_calls(nodes):
    d, Hq, Hkv = 128, 8, 2
    lens, count = [1000, 260, 77], [nodes] * 3
    cache, table = make(lens, 16, 64, Hkv, d)
    off, seen = offsets_of(count), trees_of(count)
    row = torch.zeros(off[-1], Hq + 2 * Hkv, d, dtype=torch.bfloat16).cuda()
    q = queries(off[-1], Hq, d)
    row[:, :Hq] = q
    a = check(row[:, :Hq], cache, table, lens, off, seen, d, max_q=nodes, kd=0.25, vd=4.0)
    b = ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), ints(tree.bits(seen)), max_q=nodes,
                        k_descale=0.25, v_descale=4.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # two calls at once on two streams, and a captured one replayed on other inputs
    args = (ints(table), ints(lens), ints(off), ints(tree.bits(seen)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = ea.kv4_tree_fwd(q, cache, *args, max_q=nodes, k_descale=0.25, v_descale=4.0)
    e = ea.kv4_tree_fwd(q, cache, *args, max_q=nodes, k_descale=0.25, v_descale=4.0)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c[0], b[0]) and torch.equal(e[0], b[0]) and torch.equal(c[1], b[1])
    graph, qs = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        g = ea.kv4_tree_fwd(qs, cache, *args, max_q=nodes, k_descale=0.25, v_descale=4.0)
    qs.copy_(q)
    graph.replay()
    assert torch.equal(g[0], b[0]) and torch.equal(g[1], b[1])


def test_a_chain_agrees_with_the_causal_call():
    """A chain of nodes is kv4_fwd's causal mask: both lie within the tolerances of the same reference."""
    d, lens, nodes = 128, [700, 64, 130], [6, 3, 8]
    cache, table = make(lens, 11, 64, 2, d)
    parents = [i - 1 for n in nodes for i in range(n)]
    off = offsets_of(nodes)
    seen = tree.tree_plan(parents, off, [0] * 3, 1)[1]
    q = queries(sum(nodes), 8, d)
    check(q, cache, table, lens, off, seen, d)
    check(q, cache, table, lens, off, seen, d,
          got=ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints(off), max_q=8))


def test_attention_refusals():
    cache, table = make([40], 3, 16, 2, 128)
    q, seen = queries(4, 4, 128), ints([[1], [3], [5], [9]])
    args = dict(q=q, cache=cache, table=ints(table), lens=ints([40]), q_offsets=ints([0, 4]), seen=seen)
    ea.kv4_tree_fwd(**args)
    long = ints(np.zeros((1, 400)))
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., ::2]), dict(seen=seen[:3]), dict(seen=seen[:, 0]),
                dict(seen=ints(np.zeros((4, 9)))), dict(seen=seen.cpu()), dict(seen=seen.long()),
                dict(q_offsets=ints([0, 4, 4])), dict(lens=ints([40, 1])), dict(table=ints(table)[0]),
                dict(out=q[:3].clone()), dict(lse=torch.zeros(4, 5).cuda()), dict(status=torch.zeros(1).cuda())):
        with pytest.raises(ValueError):
            ea.kv4_tree_fwd(**(args | bad))
    for bad in (dict(out=q), dict(scale=-1.0), dict(k_descale=3.0), dict(max_q=0),
                dict(table=long, workspace=torch.zeros(64, dtype=torch.uint8).cuda())):
        with pytest.raises(ea.AttentionError):
            ea.kv4_tree_fwd(**(args | bad))
    empty = ea.kv4_tree_fwd(q[:0], cache, ints(table), ints([40]), ints([0, 0]), seen[:0])
    assert empty[0].shape == (0, 4, 128)


# --------------------------------------------------------------------------------- offsets that make no sense
ODD_OFFSETS = [[0, -3, 900, 2], [5, 1, 4, 9], [2 ** 31 - 1, 0, 2, 4], [-2 ** 31, 3, 3, 2 ** 31 - 1], [4, 60, 61, 70]]


def guarded(*shape, dtype=torch.int32, guard=1 << 16):
    """A tensor of 7s in the middle of a larger one, and whether what lies on its two sides is still all 7s."""
    n = math.prod(shape)
    whole = torch.full((n + 2 * guard,), 7, dtype=dtype, device="cuda")
    return whole[guard:guard + n].view(shape), lambda: bool((whole[:guard] == 7).all() and (whole[guard + n:] == 7).all())


@pytest.mark.parametrize("off", ODD_OFFSETS)
@pytest.mark.parametrize("T", [1, 4, 60, 700])
def test_odd_offsets_write_plans_and_acceptances_nowhere_else(off, T):
    """... and nothing of a request that the offsets leave without rows."""
    lens, new, words = ints([5, 6, 90]), ints([9, 6, 95]), 2
    p = ints(random_trees(np.random.default_rng(T), [T]))
    (positions, safe_p), (seen, safe_s) = guarded(T), guarded(T, words)
    ea.tree_plan(p, ints(off), lens, 64, out=ea.TreePlan(positions, seen))
    assert safe_p() and safe_s()
    outs, safe = zip(*(guarded(n) for n in (3, 3, T, 3, T, 2)))
    queue, safe_q = guarded(40)
    ea.tree_accept(p, seen, ints([1] * T), ints([1] * T), lens, new, ints(off), ints(range(T)), ints(np.zeros((3, 6))),
                   queue, ints([38, 1]), 16, out=ea.TreeAccept(*outs))
    assert all(f() for f in safe) and safe_q()
    rows = np.zeros(T, dtype=bool)  # of some request, or behind the last one
    for first, last in [*zip(off, off[1:]), (off[-1], T)]:
        rows[max(0, min(first, T)):max(0, min(last, T))] = True
    for t in (positions, seen, outs[2], outs[4]):
        assert bool((t.cpu()[~torch.from_numpy(rows)] == 7).all())
    for b in range(3):
        n = max(0, min(off[b + 1], T) - max(0, min(off[b], T)))
        assert 0 <= int(outs[1][b]) <= n
    cache, safe_c = guarded(50, 2, 2, 16 * 36, dtype=torch.uint8)
    ea.kv4_move(cache, ints(range(T)[::-1]), ints(range(T)), ints(off), ints([2 ** 31 - 1, -1, 3]), 64)
    assert safe_c()


@pytest.mark.parametrize("off", ODD_OFFSETS)
@pytest.mark.parametrize("nodes", [1, 8, 16, 20, 50])  # units of 8, 16, 32, 64 and 256 rows
@pytest.mark.parametrize("T", [4, 60])
def test_odd_offsets_write_attention_nowhere_else(off, nodes, T):
    d, lens = 128, [300, 170, 90]
    cache, table = make(lens, 19, 16, 2, d)
    q, seen = queries(T, 4, d), ints(np.full((T, 2), -1))
    (o, safe_o), (lse, safe_l) = guarded(T, 4, d, dtype=torch.bfloat16), guarded(T, 4, dtype=torch.float32)
    size = ea.kv4_tree_workspace_bytes(4, 2, d, nodes, 16, 19)
    ws, safe_w = guarded(size, dtype=torch.uint8)
    ea.kv4_tree_fwd(q, cache, ints(table), ints(lens), ints(off), seen, max_q=nodes, out=o, lse=lse,
                    workspace=ws if size else None)
    assert safe_o() and safe_l() and safe_w()
    rows = torch.zeros(T, dtype=torch.bool)
    for first, last in zip(off, off[1:]):
        rows[max(0, min(first, T)):max(0, min(last, T))] = True
    assert bool((o.cpu()[~rows] == 7).all()) and bool((lse.cpu()[~rows] == 7).all())
    # (offsets of 900 nodes before 170 keys: the keys are nodes 730 and later, which have no bits, and no row sees any)
    assert bool(torch.isfinite(o.cpu()[rows]).all()) and bool((lse.cpu()[rows] < 1e3).all())


# --------------------------------------------------------------------------------- all of them together
@pytest.mark.parametrize("B,Hq", [(5, 4), (70, 16)])  # acceptance by one kernel and by two; 16 and 64 rows
def test_a_captured_step_on_another_stream(B, Hq):
    """Plan, rotation, append, attention, acceptance and moves of a step, captured once on a side stream and replayed with
    other trees, tokens and lengths: the same bits as the calls one by one."""
    d, page, Hkv, width, T = 64, 16, 1, 8, 4 * B + 3
    turns, _ = ea.rope_turns(d)
    axes = ea.rope_axis_pairs((8, 12, 12))
    slots = [b * width + i for b in range(B) for i in range(width)]

    def fresh(seed):
        r = np.random.default_rng(seed)
        nodes = r.integers(0, 5, B).tolist()
        lens = r.integers(1, 90, B).tolist()
        parents = random_trees(r, nodes) + [0] * (T - sum(nodes))
        return dict(nodes=ints(nodes), lens=ints(lens), parents=ints(parents), tokens=ints(r.integers(0, 2, T)),
                    choices=ints(r.integers(0, 2, T)), q=queries(T, Hq, d, seed), k=queries(T, Hkv, d, seed + 1),
                    v=queries(T, Hkv, d, seed + 2), cache=torch.randint(0, 40, (B * width + 1, Hkv, 2, page * 9 * d // 16),
                                                                        dtype=torch.uint8).cuda(),
                    table=ints(slots).view(B, width), queue=ints(np.zeros(B * width)), state=ints([0, 0]))

    def step(x):
        new = torch.minimum(x["nodes"], x["lens"] * 0 + 4)
        offsets = torch.cat([x["nodes"][:1] * 0, torch.cumsum(new, 0).int()])
        tp = ea.tree_plan(x["parents"], offsets, x["lens"], 4)
        after = x["lens"] + new
        row = torch.arange(T, device="cuda", dtype=torch.int32)
        req = torch.searchsorted(offsets[1:].contiguous(), row, right=True).clamp(max=B - 1)
        at = x["lens"][req] + row - offsets[req]
        place = torch.where(row < offsets[-1], x["table"].view(-1)[req * width + (at // page).clamp(0, width - 1)] * page
                            + at % page, -1).int()
        q, k = ea.rope_axes(x["q"], x["k"], tp.positions.expand(3, T).contiguous(), turns, axes)
        ea.kv4_append(k, x["v"], x["cache"], place)
        o, lse = ea.kv4_tree_fwd(q, x["cache"], x["table"], after, offsets, tp.seen, max_q=4)
        got = ea.tree_accept(x["parents"], tp.seen, x["tokens"], x["choices"], x["lens"], after, offsets, place,
                             x["table"], x["queue"], x["state"], page)
        ea.kv4_move(x["cache"], got.sources, place, offsets, got.counts, d)
        n = offsets[-1]
        live = (row < n)[:, None]
        return [tp.positions, tp.seen, torch.where(live[..., None], o, 0), torch.where(live, lse, 0), *got, x["cache"],
                x["queue"]]

    side = torch.cuda.Stream()
    held = fresh(100)
    with torch.cuda.stream(side):
        step({k: v.clone() for k, v in held.items()})  # (lazy initialisations)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step(held)
    for seed in (1, 2, 3):
        x = fresh(seed)
        want = step({k: v.clone() for k, v in x.items()})
        for k, v in x.items():
            held[k].copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(outs, want):
            assert torch.equal(g, w)


def test_steps_that_check_trees():
    """Four steps of three requests, each: pages, tree, positions, append, attention, acceptance, moves.  The cache
    must end up as if the accepted tokens had been written alone, one after the other, and lengths, pages and the
    ring stay consistent; attention of each step lies within the reference's tolerances."""
    d, page, Hq, Hkv, width, B, layers = 128, 16, 8, 2, 8, 3, 2
    rng = np.random.default_rng(11)
    turns, _ = ea.rope_turns(d)
    axes = ea.rope_axis_pairs((16, 24, 24))
    cap = B * width + 4
    caches = [ea.kv4_cache(cap, Hkv, page, d) for _ in range(layers)]
    table, queue = ints(np.zeros((B, width))), ints(rng.permutation(cap))
    lens, state = ints([0] * B), ints([0, cap])
    alone = [[], [], []]  # accepted keys and values of each request: rows after rotation
    accepted = 0
    for step in range(5):
        nodes = [70, 20, 45] if step == 0 else rng.integers(1, 40, B).tolist()  # first the prompts, as chains
        off = offsets_of(nodes)
        parents = [i - 1 for n in nodes for i in range(n)] if step == 0 else random_trees(rng, nodes, 3)
        T = off[-1]
        q, k, v = (normal(T, h, d, seed=100 * step + h).bfloat16().cuda() for h in (Hq, Hkv, Hkv + 1))
        v = v[:, :Hkv]
        plan = ea.page_plan(lens, ints(nodes), table, queue, state, page, T)
        assert bool((plan.slots >= 0).all())
        up = ints(parents)
        got = ea.tree_plan(up, plan.q_offsets, lens, max_nodes=max(nodes))
        pos = got.positions.expand(3, -1).contiguous()
        qr, kr = ea.rope_axes(q, k, pos, turns, axes)
        same = ea.rope(q, k, got.positions, turns)
        assert torch.equal(qr, same[0]) and torch.equal(kr, same[1])
        for cache in caches:
            ea.kv4_append(kr, v, cache, plan.slots)
        o, lse = ea.kv4_tree_fwd(qr, caches[0], table, plan.lens, plan.q_offsets, got.seen, max_q=max(nodes))
        words = got.seen.shape[1]
        seen = tree.tree_plan(parents, off, [0] * B, words)[1]
        check(qr, caches[0], table.cpu().numpy(), plan.lens.tolist(), off, seen, d, got=(o, lse))
        tokens, choices = rng.integers(0, 3, T), rng.integers(0, 3, T)
        if step == 0:
            tokens[:], choices[:] = 1, 1  # the whole prompt
        new = ea.tree_accept(up, got.seen, ints(tokens), ints(choices), lens, plan.lens, plan.q_offsets, plan.slots,
                             table, queue, plan.queue_state, page)
        ea.kv4_move(caches, new.sources, plan.slots, plan.q_offsets, new.counts, d)
        for b in range(B):
            n = int(new.counts[b])
            accepted += n > 1
            for i in new.path[off[b]:off[b] + n].tolist():
                alone[b].append((kr[off[b] + i], v[off[b] + i]))
            assert int(new.lens[b]) == len(alone[b])
        lens, state = new.lens, new.queue_state
        # every page is free or held once
        held = [p for b in range(B) for p in table[b, :-(-len(alone[b]) // page)].tolist()]
        free = [int(queue[(int(state[0]) + i) % cap]) for i in range(int(state[1]))]
        assert sorted(held + free) == list(range(cap))
    assert accepted > B
    for cache in caches:
        for b in range(B):
            n = len(alone[b])
            j = np.arange(n)
            slots = ints(table[b].cpu().numpy()[j // page] * page + j % page)
            k, v = ea.kv4_read(cache, slots, d)
            fresh = ea.kv4_cache(-(-n // page), Hkv, page, d)
            ea.kv4_append(torch.stack([x for x, _ in alone[b]]), torch.stack([x for _, x in alone[b]]), fresh, ints(j))
            k1, v1 = ea.kv4_read(fresh, ints(j), d)
            assert torch.equal(k, k1) and torch.equal(v, v1)
