"""The 4-bit cache and attention over it against the fp64 reference."""
import math

import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import kv

pytestmark = pytest.mark.gpu


def numpy64(t):
    return t.double().cpu().numpy()


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


# --------------------------------------------------------------------------------- write and read
@pytest.mark.parametrize("d,page,H,T", [(128, 16, 1, 1), (64, 16, 3, 50), (128, 64, 2, 77),
                                        (64, 128, 4, 200), (128, 32, 8, 33)])
@pytest.mark.parametrize("kd,vd", [(1.0, 1.0), (0.25, 2.0 ** -6)])
def test_append_and_read_are_exact(d, page, H, T, kd, vd):
    pages = -(-2 * T // page)
    cache = ea.kv4_cache(pages, H, page, d)
    cache.random_(0, 256, generator=torch.Generator("cuda").manual_seed(1))
    before = cache.clone()
    row = (normal(T, 2 * H, d) * torch.logspace(-3, 3, d)).bfloat16()
    row[0, 0] = 0
    row[T // 2, 1, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6] * 2)  # ties
    row = row.cuda()
    k, v = row[:, :H], row[:, H:]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:T].int()
    slots[T // 3] = -1
    if T > 5:
        slots[5] = pages * page  # the first slot past the cache
    ea.kv4_append(k, v, cache, slots.cuda(), kd, vd)
    ko, vo = ea.kv4_read(cache, slots.cuda(), d, kd, vd)
    touched = np.zeros(cache.shape, dtype=bool)
    for x, y, n, ds in ((k, ko, 0, kd), (v, vo, 1, vd)):
        code, s8 = kv.quantise(numpy64(x), ds)
        want = kv.dequantise(code, s8, ds)
        for t, s in enumerate(slots.tolist()):
            if not 0 <= s < pages * page:
                assert (y[t] == 0).all()
                continue
            assert np.array_equal(numpy64(y[t]), want[t])
            p, i = divmod(s, page)
            for h in range(H):
                raw = cache[p, h, n].cpu().numpy()
                c, sc = kv.unblock(raw, page, d)
                assert np.array_equal(c[i], code[t, h]) and np.array_equal(sc[i], s8[t, h])
            touched[p, :, n, i * d // 2:(i + 1) * d // 2] = True
            at = page * d // 2 + i * d // 16
            touched[p, :, n, at:at + d // 16] = True
    same = (cache == before).cpu().numpy()
    assert same[~touched].all()  # nothing beside the rows was written


def test_more_rows_than_one_launch_takes():
    """2^24 + 5 tokens of 8 heads are more than 2^30 pieces: the last five go in a second launch."""
    T, H, d, page = 2 ** 24 + 5, 8, 128, 16
    cache = ea.kv4_cache(2, H, page, d)
    rows = normal(1, H, d).bfloat16().cuda()
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[0], slots[-3], slots[-1] = 4, 30, 17
    ea.kv4_append(rows.expand(T, H, d), rows.expand(T, H, d), cache, slots)
    small = ea.kv4_cache(2, H, page, d)
    ea.kv4_append(rows.expand(3, H, d).contiguous(), rows.expand(3, H, d).contiguous(), small, ints([4, 30, 17]))
    assert torch.equal(cache, small) and bool(cache.any())


def test_extreme_values():
    d, page = 128, 16
    cache = ea.kv4_cache(1, 1, page, d)
    x = normal(8, 1, d).bfloat16()
    x[0] *= 1e-4           # below e4m3's smallest scale: zeros
    x[1] *= 1e37           # saturates at 448 * 6
    x[2, 0, 100] = math.nan
    x[3, 0, 0] = -math.inf
    x[4] = 6 * 448
    x[5] = -0.0
    slots = torch.arange(8, dtype=torch.int32).cuda()
    ea.kv4_append(x.cuda(), x.cuda(), cache, slots)
    k, v = ea.kv4_read(cache, slots, d)
    want = kv.dequantise(*kv.quantise(numpy64(x)))
    for y in (k, v):
        assert np.array_equal(numpy64(y), want, equal_nan=True)
    assert (want[0] == 0).all() and np.abs(want[1]).max() == 2688 and np.isnan(want[2:4]).all()


# --------------------------------------------------------------------------------- attention
def make(lens, width, page, Hkv, d, seed=0, extra=3):
    """A cache of normal keys and values with scattered pages, and its table.  Bytes that no request
    owns are 0xff: NaN scales."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    pages = B * width + extra
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    cache = torch.full((pages, Hkv, 2, page * 9 * d // 16), 255, dtype=torch.uint8).cuda()
    slots, n = [], 0
    for b, m in enumerate(lens):
        j = np.arange(max(0, min(m, width * page)))
        slots += (table[b, j // page] * page + j % page).tolist()
    if slots:
        k, v = normal(len(slots), Hkv, d, seed=seed + 1), normal(len(slots), Hkv, d, seed=seed + 2)
        k[:, :, 3] *= 6
        ea.kv4_append(k.bfloat16().cuda(), v.bfloat16().cuda(), cache, ints(slots))
    return cache, table


def check(q, cache, table, lens, offsets, d, causal=True, scale=None, kd=1.0, vd=1.0, got=None, **kw):
    """Tolerances.  A score is a sum of exact products in fp32 (d roundings at most, some by
    truncation) of queries rounded 2^-25 of the row's largest value: off by delta = 2^-18 scale
    sum|q k| at most.  p then is off by delta relative, f16 P by 2^-11 relative or, where it is
    subnormal, half of 2^-24 absolute with the row's largest P at 2^7 or more (2^-32 of it: sum p
    is at least the largest, so O is off by 2^-32 sum |v|), ex2 by 2^-21, and O = sum p v / sum p by
    the relative part twice over; bf16 O by 2^-8.  LSE is off by delta and fp32 roundings of a few 2^-22 (1 + |LSE|)."""
    scale = 1 / math.sqrt(d) if scale is None else scale
    q64 = numpy64(q)
    o64, lse64, mass, total, dot = kv.kv4_attention(q64, cache.cpu().numpy(), np.asarray(table), lens, offsets,
                                             d, scale, causal, kd, vd)
    if got is None:
        got = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints(offsets), causal=causal,
                         scale=scale, k_descale=kd, v_descale=vd, **kw)
    o, lse = (numpy64(t) for t in got)
    n = offsets[-1]
    delta = 2.0 ** -18 * scale * dot[:n]
    tol = 2.0 ** -8 * np.abs(o64[:n]) + (2 * delta[..., None] + 2.0 ** -10) * mass[:n] + 2.0 ** -32 * total[:n]
    finite = np.isfinite(lse64[:n])
    assert (np.abs(o[:n] - o64[:n]) <= tol).all(), np.nanmax(np.abs(o[:n] - o64[:n]) / tol)
    assert np.array_equal(np.isneginf(lse[:n]), ~finite)
    err = np.abs(lse[:n] - np.where(finite, lse64[:n], 0))[finite]
    lim = (delta + 2.0 ** -20 * (1 + np.abs(np.where(finite, lse64[:n], 0))))[finite]
    assert (err <= lim).all(), (err / lim).max()
    return got


def queries(T, Hq, d, seed=9):
    return (normal(T, Hq, d, seed=seed) * 2).bfloat16().cuda()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (8, 2), (7, 1), (24, 2)])
def test_decode_lengths(d, page, Hq, Hkv):
    lens = [1, 0, 15, 16, 17, 31, 33, 127, 128, 129, 300, 500]
    width = -(-500 // page)
    cache, table = make(lens, width, page, Hkv, d)
    check(queries(len(lens), Hq, d), cache, table, lens, list(range(len(lens) + 1)), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv,qlens", [
    (4, 1, [2, 0, 1, 3, 4]), (4, 4, [9, 1, 7, 8, 16]), (6, 2, [1, 5, 2, 0, 6]),
    (3, 1, [40, 3, 20, 1, 64]), (16, 2, [130, 2, 33, 5, 1]),
])
def test_several_queries_per_request(d, causal, Hq, Hkv, qlens):
    """Row blocks of 8, 16 and 32, several of them, rows before the cache's first key."""
    lens = [130, 64, 5, 0, 333]
    cache, table = make(lens, 6, 64, Hkv, d)
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    check(queries(offsets[-1], Hq, d), cache, table, lens, offsets, d, causal=causal,
          max_q=max(qlens))
    check(queries(offsets[-1], Hq, d), cache, table, lens, offsets, d, causal=causal, max_q=1)


@pytest.mark.parametrize("d,page,lens,qlens,Hq,Hkv", [
    (128, 64, [20000], [1], 8, 1), (64, 16, [9000, 3], [2, 1], 4, 1),
    (128, 128, [5000, 0, 7001, 1], [1, 1, 3, 1], 10, 2), (128, 32, [30000], [8], 4, 1),
])
def test_long_caches_split_over_the_gpu(d, page, lens, qlens, Hq, Hkv):
    cache, table = make(lens, -(-max(lens) // page), page, Hkv, d)
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    q = queries(offsets[-1], Hq, d)
    size = ea.kv4_workspace_bytes(Hq, Hkv, d, max(qlens), page, table.shape[1])
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    a = check(q, cache, table, lens, offsets, d, max_q=max(qlens), workspace=ws)
    b = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints(offsets), max_q=max(qlens),
                   workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits again


def test_many_short_requests():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 70, 700).tolist()
    cache, table = make(lens, 5, 16, 1, 64)
    check(queries(700, 2, 64), cache, table, lens, list(range(701)), 64)


def check_on_gpu(q, cache, table, lens, offsets, d, causal=True, kd=1.0, vd=1.0, **kw):
    """As ``check``, with the fp64 reference computed by torch on the GPU (large shapes); pages that
    are not in the cache hold keys that nobody sees."""
    scale = 1 / math.sqrt(d)
    pages, Hkv = cache.shape[:2]
    page, group = cache.shape[3] * 16 // (9 * d), q.shape[1] // Hkv
    raw = cache.cpu().numpy()
    o, lse = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints(offsets), causal=causal,
                        k_descale=kd, v_descale=vd, **kw)
    for b, n in enumerate(lens):
        rows = offsets[b + 1] - offsets[b]
        if rows == 0:
            continue
        if n == 0:
            assert (o[offsets[b]:offsets[b + 1]] == 0).all()
            assert (lse[offsets[b]:offsets[b + 1]] == -math.inf).all()
            continue
        ids = [int(p) for p in np.asarray(table)[b, :-(-n // page)]]
        there = torch.tensor([0 <= p < pages for p in ids]).repeat_interleave(page)[:n].cuda()
        kv64 = []
        for kind, ds in ((0, kd), (1, vd)):
            blocks = [[kv.dequantise(*kv.unblock(raw[p if 0 <= p < pages else 0, h, kind], page, d), ds)
                       for p in ids] for h in range(Hkv)]
            kv64.append(torch.tensor(np.stack([np.concatenate(x) for x in blocks]))[:, :n].cuda())
        k, v = (x.repeat_interleave(group, 0) for x in kv64)  # [Hq, n, d]
        x = q[offsets[b]:offsets[b + 1]].double().transpose(0, 1)
        s = scale * x @ k.transpose(1, 2)
        seen = there[None].expand(rows, n)
        if causal:
            seen = seen & (torch.arange(n, device="cuda")[None]
                           <= n - rows + torch.arange(rows, device="cuda")[:, None])
        s = s.masked_fill(~seen, -math.inf)
        want_l = torch.logsumexp(s, -1)
        p = torch.where(want_l[..., None] > -math.inf, torch.exp(s - want_l[..., None]), 0.0)
        want_o, mass = p @ v, p @ v.abs()
        dot = scale * (x.abs() @ k.abs().transpose(1, 2)).amax(-1)
        total = v.abs().sum(1)[:, None]
        got_o = o[offsets[b]:offsets[b + 1]].double().transpose(0, 1)
        got_l = lse[offsets[b]:offsets[b + 1]].double().T
        delta = 2.0 ** -18 * dot
        tol = 2.0 ** -8 * want_o.abs() + (2 * delta[..., None] + 2.0 ** -10) * mass + 2.0 ** -32 * total
        assert ((got_o - want_o).abs() <= tol).all()
        dead = want_l == -math.inf
        assert torch.equal(got_l == -math.inf, dead)
        err = (got_l - want_l).abs()[~dead]
        assert (err <= (delta + 2.0 ** -20 * (1 + want_l.abs()))[~dead]).all()
    return o, lse


@pytest.mark.parametrize("d,page,Hq,Hkv,lens,qlens,causal", [
    (128, 64, 8, 2, [1500, 700, 300], [700, 33, 300], True),   # rows that see nothing but themselves
    (64, 16, 4, 1, [2000, 65], [1000, 65], True),
    (128, 16, 4, 4, [1000, 129, 0, 640], [128, 129, 5, 257], False),
    (64, 128, 6, 2, [900, 1, 50], [90, 1, 60], True),          # more queries than keys
    (128, 32, 32, 1, [513], [9], True),                        # few tokens, many heads of one group
    (128, 128, 16, 16, [400] * 12, [130] * 12, True),          # more units than CTAs: several in a row
])
def test_prompt_chunks(d, page, Hq, Hkv, lens, qlens, causal):
    cache, table = make(lens, -(-max(lens) // page) + 1, page, Hkv, d)
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    q = queries(offsets[-1], Hq, d)
    a = check_on_gpu(q, cache, table, lens, offsets, d, causal=causal, max_q=max(qlens), vd=0.5)
    b = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints(offsets), causal=causal,
                   max_q=max(qlens), v_descale=0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits again
    assert ea.device_status() == 0


def test_prompt_chunk_split_over_many_ctas():
    """One key head and two blocks of rows: every CTA takes a few tiles, all of them are merged."""
    d, page, lens, qlens = 128, 64, [20000], [100]
    cache, table = make(lens, 313, page, 1, d)
    size = ea.kv4_workspace_bytes(4, 1, d, 100, page, 313)
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    check_on_gpu(queries(100, 4, d), cache, table, lens, [0, 100], d, max_q=100, workspace=ws)


def test_prompt_chunks_with_masked_places_and_missing_pages():
    d, page, lens, qlens = 64, 32, [700, 300], [200, 90]
    cache, table = make(lens, 22, page, 2, d)
    offsets = [0, 200, 290]
    q = queries(290, 4, d)
    want = check_on_gpu(q, cache, table, lens, offsets, d, max_q=200)
    # the key of request 0's query 150 becomes NaN: queries before it do not see it
    at = 700 - 200 + 150
    slot = ints([table[0][at // page] * page + at % page])
    bad = torch.full((1, 2, d), math.nan).bfloat16().cuda()
    good_k, good_v = ea.kv4_read(cache, slot, d)
    for k, v in ((bad, good_v), (good_k, bad)):
        ea.kv4_append(k, v, cache, slot)
        o, lse = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints(offsets), max_q=200)
        sees = torch.zeros(290, dtype=torch.bool)
        sees[150:200] = True
        assert torch.equal(o[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees])
        assert o[sees].isnan().all() and lse[sees].isnan().all()
    ea.kv4_append(good_k, good_v, cache, slot)
    table[0, 3], table[0, 20], table[1, 0], table[1, 9] = -1, 2 ** 31 - 1, -7, 10 ** 6
    check_on_gpu(q, cache, table, lens, offsets, d, max_q=200)


@pytest.mark.parametrize("d,B", [(64, 1200), (128, 545)])
def test_many_requests_of_few_rows_as_chunks(d, B):
    """``max_q`` only picks the kernel: more requests than a CTA has threads, most of a token or two,
    some without tokens or keys, one long."""
    rng = np.random.default_rng(B)
    lens, qlens = rng.integers(0, 40, B), rng.integers(0, 3, B)
    lens[B // 2], qlens[B // 2] = 900, 70
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    cache, table = make(lens.tolist(), 57, 16, 2, d)
    check(queries(offsets[-1], 4, d), cache, table, lens.tolist(), offsets, d, max_q=70)


def test_a_cache_of_more_than_4_gb():
    """The same bits from pages past 2^32 bytes as from a small cache."""
    d, page, Hq, Hkv, lens = 128, 128, 16, 8, [700, 200]
    qlens = [3, 40]
    width, offsets = 6, ints([0, 3, 43])
    pages = 2 ** 32 // (2 * Hkv * page * 72) + 50
    big = torch.empty((pages, Hkv, 2, page * 72), dtype=torch.uint8, device="cuda")
    small = ea.kv4_cache(2 * width, Hkv, page, d)
    high = torch.arange(pages - 2 * width, pages).view(2, width).flip(0)
    assert int(high.min()) * 2 * Hkv * page * 72 > 2 ** 32
    q, res = queries(43, Hq, d), []
    for cache, table in ((small, torch.arange(2 * width).view(2, width)), (big, high)):
        slots = torch.cat([table[b][torch.arange(n) // page] * page + torch.arange(n) % page
                           for b, n in enumerate(lens)])
        k, v = (normal(sum(lens), Hkv, d, seed=i).bfloat16().cuda() for i in (1, 2))
        ea.kv4_append(k, v, cache, ints(slots))
        res.append([*ea.kv4_read(cache, ints(slots), d)])
        for max_q in (1, 4, 8, 40):
            res[-1] += ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=offsets, max_q=max_q)
    for x, y in zip(*res):
        assert torch.equal(x, y)
    assert not res[0][2].isnan().any()


def test_prompts_of_many_blocks():
    """One prompt of 50 and one of 7 blocks of rows between short ones, on more and fewer key heads."""
    d, page, lens, qlens = 64, 64, [90, 3300, 70, 800, 40], [40, 3200, 70, 440, 33]
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    for Hq, Hkv in ((4, 1), (4, 2)):
        cache, table = make(lens, 52, page, Hkv, d)
        check_on_gpu(queries(offsets[-1], Hq, d), cache, table, lens, offsets, d, max_q=3200)


def test_prompt_chunks_at_once_captured_and_rows_outside():
    """Calls of both kernels on two streams at once; a graph replayed on new data; rows before the
    first request's and past the last one's are left as they are."""
    d, page, Hq, Hkv, lens, qlens = 128, 32, 8, 2, [900, 200], [150, 40]
    cache, table = make(lens, 29, page, Hkv, d)
    offsets, tab, ln = ints([2, 152, 192]), ints(table), ints(lens)
    q = queries(200, Hq, d)
    q[:2] = math.nan
    q[192:] = math.nan
    want = check_on_gpu(q[2:192].contiguous(), cache, table, lens, [0, 150, 190], d, max_q=150)
    dec_q = queries(2, Hq, d, seed=3)
    dec = ea.kv4_fwd(dec_q, cache, tab, ln)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(s):
            for _ in range(3):
                o = torch.full((200, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
                lse = torch.full((200, Hq), 8.0, device="cuda")
                ea.kv4_fwd(q, cache, tab, ln, q_offsets=offsets, max_q=150, out=o, lse=lse)
                got.append((o, lse, ea.kv4_fwd(dec_q, cache, tab, ln)))
    torch.cuda.synchronize()
    for o, lse, x in got:
        assert torch.equal(o[2:192], want[0]) and torch.equal(lse[2:192], want[1])
        for rest in (slice(0, 2), slice(192, 200)):
            assert (o[rest] == 7).all() and (lse[rest] == 8).all()
        assert torch.equal(x[0], dec[0]) and torch.equal(x[1], dec[1])
    static = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ea.kv4_fwd(static, cache, tab, ln, q_offsets=offsets, max_q=150)
    for sign in (1, -1):
        static.copy_(sign * q)
        graph.replay()
        eager = ea.kv4_fwd(static, cache, tab, ln, q_offsets=offsets, max_q=150)
        assert torch.equal(o[2:192], eager[0][2:192]) and torch.equal(lse[2:192], eager[1][2:192])
    assert ea.device_status() == 0


def test_scale_descales_and_large_scores():
    lens, d = [200, 77], 128
    cache, table = make(lens, 4, 64, 2, d)
    q = queries(2, 4, d)
    for scale, kd, vd in ((0.0, 1.0, 1.0), (3.0, 1.0, 0.5), (0.02, 8.0, 2.0 ** -9)):
        check(q, cache, table, lens, [0, 1, 2], d, scale=scale * 1.0, kd=kd, vd=vd)
    big = q.clone()
    big[0, 0] *= 1e30
    big[0, 1] *= 1e-30
    big[1, 0] = 0
    check(big, cache, table, lens, [0, 1, 2], d, scale=1e-30)
    # rising scores: the running maximum moves in every strip
    k = torch.ones(200, 2, d) * torch.linspace(0.1, 6, 200)[:, None, None]
    slots = ints((np.asarray(table)[0][np.arange(200) // 64] * 64 + np.arange(200) % 64))
    ea.kv4_append(k.bfloat16().cuda(), k.bfloat16().cuda(), cache, slots)
    check(torch.ones(2, 4, d).bfloat16().cuda(), cache, table, lens, [0, 1, 2], d, scale=1.0)
    check(-torch.ones(2, 4, d).bfloat16().cuda(), cache, table, lens, [0, 1, 2], d, scale=1.0)


def test_masked_places_hold_anything():
    """NaN keys and values past a request's length and after a query's own position."""
    d, lens, qlens = 128, [100, 40], [4, 2]
    cache, table = make(lens, 2, 64, 1, d)
    q = queries(6, 2, d)
    want = check(q, cache, table, lens, [0, 4, 6], d)
    slot = ints([np.asarray(table)[0][1] * 64 + 99 - 64])  # request 0's last key: row 3 alone sees it
    bad = torch.full((1, 1, d), math.nan).bfloat16().cuda()
    good_k, good_v = ea.kv4_read(cache, slot, d)
    for k, v in ((bad, good_v), (good_k, bad)):
        ea.kv4_append(k, v, cache, slot)
        o, lse = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints([0, 4, 6]))
        rows = [0, 1, 2, 4, 5]
        assert torch.equal(o[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
        assert o[3].isnan().all() and lse[3].isnan().all()


@pytest.mark.parametrize("max_q", [1, 8, 40])
def test_infinite_and_nan_queries_stay_in_their_row(max_q):
    d, lens, qlens = 128, [300, 90], [40, 5]
    cache, table = make(lens, 5, 64, 2, d)
    offsets = [0, 40, 45]
    q = queries(45, 4, d)
    args = (cache, ints(table), ints(lens), ints(offsets))
    want = ea.kv4_fwd(q, *args, max_q=max_q)
    bad = q.clone()
    for row, head, value in ((0, 0, math.inf), (17, 3, -math.inf), (39, 1, math.nan), (44, 2, math.inf)):
        bad[row, head, 7] = value
    o, lse = ea.kv4_fwd(bad, *args, max_q=max_q)
    hit = torch.zeros(45, 4, dtype=torch.bool)
    hit[0, 0] = hit[17, 3] = hit[39, 1] = hit[44, 2] = True
    assert torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    # a score of +inf leaves no finite softmax, nor does a NaN
    assert o[hit].isnan().any(-1).all() and not lse[hit].isfinite().any()


def test_bad_device_data_is_not_followed():
    """Page ids outside the cache are keys that are not there; lengths and offsets are clamped."""
    d, lens = 64, [192, 130, 20]
    cache, table = make(lens, 3, 64, 2, d)
    table[0, 0], table[1, 1], table[2, 0] = -1, 10 ** 6, 2 ** 31 - 1
    q = queries(3, 4, d)
    check(q, cache, table, lens, [0, 1, 2, 3], d)
    huge = [2 ** 31 - 1, -5, 1]
    check(q, cache, table, huge, [0, 1, 2, 3], d)
    out = torch.full((3, 4, d), 7.0, dtype=torch.bfloat16).cuda()
    ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints([-3, 2, 1, 2 ** 31 - 1]), out=out)
    torch.cuda.synchronize()


def test_rows_past_the_last_request_stay():
    d, lens = 128, [50, 70]
    cache, table = make(lens, 2, 64, 1, d)
    q = queries(5, 2, d)
    q[3:] = math.nan
    out = torch.full((5, 2, d), 7.0, dtype=torch.bfloat16).cuda()
    lse = torch.full((5, 2), 8.0).cuda()
    got = ea.kv4_fwd(q, cache, ints(table), ints(lens), q_offsets=ints([0, 1, 3]), out=out, lse=lse)
    check(q[:3], cache, table, lens, [0, 1, 3], d, got=(got[0][:3], got[1][:3]))
    assert (out[3:] == 7).all() and (lse[3:] == 8).all()


def test_strided_queries_and_uniform_rows():
    d, lens = 64, [50, 170, 9]
    cache, table = make(lens, 3, 64, 2, d)
    wide = queries(6, 9, d)
    q = wide[:, 2:6]
    a = ea.kv4_fwd(q, cache, ints(table), ints(lens))
    b = check(q.contiguous(), cache, table, lens, [0, 2, 4, 6], d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_and_two_captured_graphs():
    d, lens = 128, [3000, 10, 500]
    cache, table = make(lens, 47, 64, 2, d)
    q = queries(3, 8, d)
    tab, ln = ints(table), ints(lens)
    want = check(q, cache, table, lens, [0, 1, 2, 3], d)
    side, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s in side:  # two calls at once, each with its own workspace
        with torch.cuda.stream(s):
            outs.append([ea.kv4_fwd(q, cache, tab, ln) for _ in range(3)])
    torch.cuda.synchronize()
    graphs, res = [], []
    ws = torch.empty(ea.kv4_workspace_bytes(8, 2, d, 1, 64, 47), dtype=torch.uint8).cuda()
    for _ in range(2):  # two graphs that share a workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(ea.kv4_fwd(q, cache, tab, ln, workspace=ws))
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        ws.fill_(255)
        g.replay()
    torch.cuda.synchronize()
    for o, lse in [x for run in outs for x in run] + res:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("captured", [False, True])
def test_kernels_that_follow_each_other_across_streams(captured):
    """plan, rope, append, read and attention, each of which may begin before the one before it has
    ended, over forks and joins of two streams: the same bits as one after the other."""
    d, page, T, Hq, Hkv = 128, 16, 300, 4, 2
    B, width = 3, 40
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width).flip(0).contiguous()
    queue, state = ints([0]), ints([0, 0])
    k, v, q = (normal(T, h, d, seed=i).bfloat16().cuda() for i, h in enumerate((Hkv, Hkv, Hq)))
    big = torch.randn(4096, 4096, device="cuda")
    turns, m = ea.rope_turns(d)
    side = torch.cuda.Stream()

    def steps(two):
        main, outs = torch.cuda.current_stream(), []
        cache = torch.zeros(B * width, Hkv, 2, page * 9 * d // 16, dtype=torch.uint8, device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        for step in range(3):
            plan = ea.page_plan(lens, lens, table, queue, state, page, T)
            slots = (torch.arange(T, dtype=torch.int32, device="cuda") * (step + 1) % (B * width * page))
            if two:
                side.wait_stream(main)
                with torch.cuda.stream(side):
                    big @ big  # something long before the queries
                    qr, _ = ea.rope(q, None, slots, turns, mscale=m)
                kr, _ = ea.rope(k, None, slots, turns, mscale=m)
                ea.kv4_append(kr, v, cache, slots)
                main.wait_stream(side)
            else:
                qr, kr = ea.rope(q, k, slots, turns, mscale=m)
                ea.kv4_append(kr, v, cache, slots)
            rk, rv = ea.kv4_read(cache, slots, d)
            o, lse = ea.kv4_fwd(qr, cache, table, torch.full((B,), 600, dtype=torch.int32, device="cuda"))
            outs += [plan.slots, plan.lens, qr, kr, rk, rv, o, lse]
        return outs

    want = [x.clone() for x in steps(False)]
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            big @ big  # the library's own workspaces, before the capture
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = steps(True)
        for _ in range(3):
            graph.replay()
    else:
        got = steps(True)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_refusals():
    d, lens = 128, [5]
    cache, table = make(lens, 50, 16, 2, d)
    q, tab, ln = queries(1, 4, d), ints(table), ints(lens)
    ok = dict(q=q, cache=cache, table=tab, lens=ln)
    for bad in (dict(q=q.float()), dict(q=queries(1, 3, d)), dict(q=queries(1, 4, 64)[..., ::2]),
                dict(cache=cache.cpu()), dict(cache=cache[:, :, :, :-16]), dict(table=tab.long()),
                dict(table=tab[0]), dict(lens=ints([1, 2])), dict(q_offsets=ints([0])),
                dict(q=queries(3, 4, d), table=ints([[0] * 50, [1] * 50]), lens=ints([1, 2])),
                dict(out=torch.empty(1, 4, d).cuda()), dict(lse=torch.empty(1, 3).cuda()),
                dict(q_offsets=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            ea.kv4_fwd(**{**ok, **bad})
    for bad in (dict(scale=-1.0), dict(k_descale=3.0), dict(max_q=0),
                dict(workspace=torch.empty(16, dtype=torch.uint8).cuda())):
        with pytest.raises((ea.AttentionError, ValueError)):
            ea.kv4_fwd(**{**ok, **bad})
    k = normal(2, 2, d).bfloat16().cuda()
    for args in ((k, k, cache, ints([0])), (k[:, :1], k[:, :1], cache, ints([0, 1])),
                 (k, k[:1], cache, ints([0, 1])), (k.float(), k.float(), cache, ints([0, 1]))):
        with pytest.raises(ValueError):
            ea.kv4_append(*args)
    with pytest.raises(ea.AttentionError):
        ea.kv4_fwd(**ok, out=q)
    with pytest.raises(ea.AttentionError):
        ea.kv4_read(cache, ints([0, 1]), d, k=k, v=k)
    with pytest.raises(ValueError):
        ea.kv4_read(cache, ints([[0]]), d)


# --------------------------------------------------------------------------------- a serving loop
@pytest.mark.parametrize("d,page,Hq,Hkv", [(128, 16, 8, 2), (64, 64, 4, 4)])
def test_a_serving_loop(d, page, Hq, Hkv):
    """plan -> rope -> append -> attention over several steps (prompt chunks, single tokens, a request
    that ends and one that starts), against the fp64 attention on the cache's own bytes, and the
    cache against the quantised fp64 keys."""
    rng = np.random.default_rng(7)
    B, width = 4, 12
    pages = B * width
    turns, m = ea.rope_turns(d, scaling="linear", factor=2.0)
    cache = ea.kv4_cache(pages, Hkv, page, d)
    table = torch.zeros(B, width, dtype=torch.int32).cuda()
    queue = ints(rng.permutation(pages))
    state, lens = ints([0, pages]), ints([0] * B)
    for step, new in enumerate([[30, 5, 0, 17], [1, 1, 20, 1], [1, 1, 1, -1], [3, 2, 1, 40], [1, 1, 1, 1]]):
        T = sum(max(n, 0) for n in new)
        plan = ea.page_plan(lens, ints(new), table, queue, state, page, T)
        q, k = queries(T, Hq, d, seed=10 + step), queries(T, Hkv, d, seed=20 + step)
        v = queries(T, Hkv, d, seed=30 + step)
        qr, kr = ea.rope(q, k, plan.positions, turns, mscale=m)
        ea.kv4_append(kr, v, cache, plan.slots)
        kc, vc = ea.kv4_read(cache, plan.slots, d)
        assert np.array_equal(numpy64(kc), kv.dequantise(*kv.quantise(numpy64(kr))))
        assert np.array_equal(numpy64(vc), kv.dequantise(*kv.quantise(numpy64(v))))
        got = ea.kv4_fwd(qr, cache, table, plan.lens, q_offsets=plan.q_offsets, max_q=max(new))
        check(qr, cache, table.cpu().numpy(), plan.lens.tolist(), plan.q_offsets.tolist(), d, got=got)
        lens, state = plan.lens, plan.queue_state
    assert lens.tolist() == [36, 10, 23, 41]


def test_a_step_without_tokens():
    """All requests end: the plan gives their pages back and the other calls, on no rows, write nothing."""
    d, page, Hq, Hkv = 128, 16, 8, 2
    cache = ea.kv4_cache(6, Hkv, page, d)
    cache.random_(0, 256, generator=torch.Generator("cuda").manual_seed(1))
    before = cache.clone()
    turns, _ = ea.rope_turns(d)
    table, queue = ints([[0, 1, 2], [3, 4, 5]]), ints([9] * 6)
    plan = ea.page_plan(ints([20, 40]), ints([-1, -1]), table, queue, ints([0, 0]), page, 0)
    assert plan.lens.tolist() == [0, 0] and plan.q_offsets.tolist() == [0, 0, 0]
    assert plan.queue_state.tolist() == [0, 5] and sorted(queue.tolist()) == [0, 1, 3, 4, 5, 9]
    q, k = queries(0, Hq, d), queries(0, Hkv, d)
    qr, kr = ea.rope(q, k, plan.positions, turns)
    assert qr.shape == q.shape and kr.shape == k.shape
    ea.kv4_append(kr, k, cache, plan.slots)
    assert [x.shape for x in ea.kv4_read(cache, plan.slots, d)] == [k.shape, k.shape]
    for kw in (dict(q_offsets=plan.q_offsets, max_q=max(-1, -1)), dict(q_offsets=plan.q_offsets, max_q=0), {}):
        o, lse = ea.kv4_fwd(qr, cache, table, plan.lens, **kw)
        assert o.shape == q.shape and lse.shape == (0, Hq)
    assert torch.equal(cache, before)
    for shape in ((2, 4, 0, d), (0, 4, 7, d)):  # training tensors of no rows
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        y, _ = ea.rope(x, x, torch.zeros(shape[2], dtype=torch.int32, device="cuda"), turns, inverse=True)
        assert y.shape == x.shape
    with pytest.raises(ValueError):
        ea.kv4_fwd(q.float(), cache, table, plan.lens)
    with pytest.raises(ValueError):
        ea.kv4_append(k, k, cache, ints([1]))


def test_calls_with_the_other_head_dim_are_refused():
    cache, slots = ea.kv4_cache(4, 2, 128, 64), ints([0])
    wide = normal(1, 2, 128).bfloat16().cuda()
    for call in (lambda: ea.kv4_read(cache, slots, 128), lambda: ea.kv4_append(wide, wide, cache, slots),
                 lambda: ea.kv4_fwd(wide, cache, ints([[0]]), ints([1]))):
        with pytest.raises(ValueError, match="made for d = 64"):
            call()
    assert ea.kv4_read(cache, slots, 64)[0].shape == (1, 2, 64)


def test_the_largest_max_q():
    """Any max_q from 1 on is correct, as documented, those past 32 bits too."""
    d, lens, qlens = 64, [300, 90], [3, 2]
    cache, table = make(lens, 5, 64, 2, d)
    for max_q in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1):
        check(queries(5, 4, d), cache, table, lens, [0, 3, 5], d, max_q=max_q)


def test_a_status_word_elsewhere_is_refused():
    """The kernel writes to it when a wait runs out: not to host memory, nor 4 bytes into fewer."""
    d, lens = 64, [70]
    cache, table = make(lens, 5, 64, 2, d)
    q, args = queries(1, 4, d), (ints(table), ints(lens))
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int16).cuda(),
                torch.zeros(0, dtype=torch.int32).cuda()):
        with pytest.raises(ValueError, match="status"):
            ea.kv4_fwd(q, cache, *args, status=bad)
    word = torch.full((1,), 7, dtype=torch.int32).cuda()
    for max_q in (1, 64):
        a = ea.kv4_fwd(q, cache, *args, max_q=max_q, status=word)
        b = ea.kv4_fwd(q, cache, *args, max_q=max_q)
        assert torch.equal(a[0], b[0]) and word.item() == 7


@pytest.mark.parametrize("captured", [False, True])
def test_each_call_waits_for_what_the_one_before_it_writes(captured):
    """plan -> rope -> rope -> append -> read -> attention -> plan -> plan ..., each on the outputs of the ones before,
    with no other kernel between them: the same bits as with a wait after every call.  All outputs hold
    other values beforehand, so a kernel that reads too early takes those."""
    d, page, Hq, Hkv, B, width = 128, 64, 16, 4, 64, 12
    rng = np.random.default_rng(11)
    news = [rng.integers(300, 500, B), np.ones(B, int), rng.integers(-1, 5, B), rng.integers(0, 9, B)]
    sizes = [int(np.maximum(n, 0).sum()) + 1 for n in news]
    new = [ints(n) for n in news]
    q, k, v = ([queries(T, h, d, seed=40 * i + s) for s, T in enumerate(sizes)]
               for i, h in enumerate((Hq, Hkv, Hkv)))
    turns, m = ea.rope_turns(d)
    queue0, big = ints(rng.permutation(B * width)), torch.randn(8192, 8192, device="cuda").bfloat16()
    work = max(ea.kv4_workspace_bytes(Hq, Hkv, d, int(n.max()), page, width) for n in news)
    bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    plan = lambda T: ea.PagePlan(*(torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
                                   for n in (B, B + 1, T, T, 2)))
    state = [torch.empty(B, width, dtype=torch.int32, device="cuda"), torch.empty_like(queue0),
             torch.empty(B * width, Hkv, 2, page * 9 * d // 16, dtype=torch.uint8, device="cuda")]
    lens0, count0, ws = ints([0] * B), ints([0, B * width]), torch.empty(work, dtype=torch.uint8, device="cuda")
    outs = [(plan(T), plan(0), bf16(T, Hq, d), bf16(T, Hkv, d), bf16(T, Hq, d), bf16(T, Hkv, d), bf16(T, Hkv, d),
             bf16(T, Hq, d), torch.empty(T, Hq, device="cuda")) for T in sizes]

    def reset():
        state[0].fill_(0)
        state[1].copy_(queue0)
        state[2].fill_(255)
        ws.fill_(255)
        for step in outs:
            for t in step:
                for x in t if isinstance(t, tuple) else (t,):
                    x.fill_(3 if x.dtype is torch.int32 else math.nan)

    def chain(wait):
        (table, queue, cache), lens, count = state, lens0, count0
        for s, (p, p2, qr, kr, qb, ko, vo, o, lse) in enumerate(outs):
            for call in (lambda: ea.page_plan(lens, new[s], table, queue, count, page, sizes[s], out=p),
                         lambda: ea.rope(q[s], k[s], p.positions, turns, mscale=m, q_out=qr, k_out=kr),
                         lambda: ea.rope(qr, None, p.positions, turns, inverse=True, q_out=qb),
                         lambda: ea.kv4_append(kr, v[s], cache, p.slots),
                         lambda: ea.kv4_read(cache, p.slots, d, k=ko, v=vo),
                         lambda: ea.kv4_fwd(qr, cache, table, p.lens, p.q_offsets, max_q=int(news[s].max()),
                                            out=o, lse=lse, workspace=ws),
                         lambda: ea.page_plan(p.lens, lens0, table, queue, p.queue_state, page, 0, out=p2)):
                call()
                if wait:
                    torch.cuda.synchronize()
            lens, count = p2.lens, p2.queue_state

    def results():
        torch.cuda.synchronize()
        flat = [x for step in outs for t in step for x in (t if isinstance(t, tuple) else (t,))]
        return [x.view(torch.uint8).clone() for x in flat + state]

    reset()
    chain(True)
    want = results()
    assert outs[-1][0].lens.sum() > 0 and not outs[0][7][:-1].isnan().any()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(False)
    for _ in range(3):
        reset()
        if captured:
            graph.replay()
        else:
            for _ in range(8):  # the host runs ahead meanwhile
                big @ big
            chain(False)
        for x, y in zip(results(), want):
            assert torch.equal(x, y)


def test_rows_on_both_sides_of_a_launch_border():
    """An append takes 2^30 / 64 tokens of 8 heads of 128 in a launch, a read 2^30 / 128: rows around those
    borders, on rows that differ (windows of one buffer, 8 values apart)."""
    H, d, page, T = 8, 128, 16, 2 ** 24 + 5
    flat = torch.randn(8 * T + 2 * H * d, device="cuda").bfloat16()
    k = flat.as_strided((T, H, d), (8, 128, 1))
    v = flat[8:].as_strided((T, H, d), (8, 64, 1))
    at = [0, 2 ** 23 - 1, 2 ** 23, 2 ** 23 + 1, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, T - 1]
    where = torch.tensor(at).cuda()
    cache, small = ea.kv4_cache(2, H, page, d), ea.kv4_cache(2, H, page, d)
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    own = ints([4, 30, 17, 0, 9, 31, 2, 16])
    slots[where] = own
    ea.kv4_append(k, v, cache, slots)
    ea.kv4_append(k[where].contiguous(), v[where].contiguous(), small, own)
    assert torch.equal(cache, small) and len({bytes(x) for x in small[:, 0, 0].cpu().numpy()}) == 2
    want = ea.kv4_read(small, own, d)
    T = 2 ** 23 + 9  # two launches
    slots = slots[:T].contiguous()
    got = ea.kv4_read(cache, slots, d)
    inside = where[where < T]
    for x, y in zip(got, want):
        assert torch.equal(x[inside], y[:len(inside)])
        x[inside] = 0
        assert not any(bool(part.view(torch.int32).any()) for part in x.split(2 ** 20))
    del got, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,max_q,Hq", [(129, 1, 4), (300, 1, 4), (129, 8, 2), (300, 8, 4)])
def test_more_requests_than_threads_with_split_units(d, B, max_q, Hq):
    """The line of work found in pieces of 128 requests, beside units that cross CTAs: lengths of nothing
    to thousands, requests without queries."""
    rng = np.random.default_rng(B + max_q)
    page, width = 32, 130
    lens = rng.integers(0, 200, B)
    lens[rng.integers(0, B, 6)] = 0
    lens[[3, 127, 128, B - 1]] = 4100, 1, 3000, 2500
    qlens = rng.integers(0, max_q + 1, B)
    qlens[[3, 127, 128, B - 1]] = max_q
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    cache, table = make(lens.tolist(), width, page, 1, d)
    size = ea.kv4_workspace_bytes(Hq, 1, d, max_q, page, width)
    assert size > 0
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    check_on_gpu(queries(offsets[-1], Hq, d), cache, table, lens.tolist(), offsets, d, max_q=max_q, workspace=ws)


def test_strides_past_32_bits():
    """Queries, keys and values whose rows lie 2^26 values apart: the last ones beyond 2^32."""
    d, page, Hq, Hkv, T, far = 64, 16, 4, 2, 70, 2 ** 26
    flat = torch.empty((T - 1) * far + (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device="cuda")
    rows = flat.as_strided((T, Hq + 2 * Hkv, d), (far, d, 1))
    near = queries(T, Hq + 2 * Hkv, d)
    rows.copy_(near)
    turns, _ = ea.rope_turns(d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    res = []
    for x in (near, rows):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        cache = ea.kv4_cache(5, Hkv, page, d)
        ea.rope(q, k, pos, turns, q_out=q, k_out=k)
        ea.kv4_append(k, v, cache, pos)
        res.append([q.clone(), k.clone(), cache])
        for max_q in (1, 8, T):
            res[-1] += ea.kv4_fwd(q, cache, pos[None, :5].contiguous(), ints([T]), max_q=max_q)
    for x, y in zip(*res):
        assert torch.equal(x, y)
    del flat, rows, q, k, v, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d,max_q,qlens,T", [(64, 1, [2, 9, 3], 7), (128, 8, [2, 8, 3], 3), (128, 4, [3, 8, 3], 12),
                                             (128, 150, [40, 150, 60], 150), (64, 150, [40, 150, 60], 245)])
def test_a_batch_cut_short_keeps_its_rows_places(d, max_q, qlens, T):
    """A plan of fewer tokens than the requests bring: the rows that there are see the keys up to their own, not
    those of the rows cut off."""
    lens = [130, 400, 90]
    cache, table = make(lens, 8, 64, 2, d)
    offsets = np.concatenate([[0], np.cumsum(qlens)]).tolist()
    assert T < offsets[-1]
    q = queries(offsets[-1], 4, d)
    check(q[:T].contiguous(), cache, table, lens, offsets, d, max_q=max_q)
    check(q, cache, table, lens, offsets, d, max_q=max_q)
