"""The fp64 reference of the operators around attention, pinned against the mathematics (CPU only)."""
import math

import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import kv


def test_small_float_grids():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(kv.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())
    assert kv.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def test_nearest_is_round_to_even():
    x = torch.linspace(0, 460, 100001, dtype=torch.float64)
    want = x.clamp(max=448).float().to(torch.float8_e4m3fn).double().numpy()
    # fp32 and fp64 agree on these points except where fp32's own rounding reaches a midpoint
    exact = x.float().double().numpy()
    assert np.array_equal(kv.E4M3[kv.nearest(exact, kv.E4M3)], want)
    mid = (kv.E2M1[1:] + kv.E2M1[:-1]) / 2
    assert kv.E2M1[kv.nearest(mid, kv.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4]
    assert kv.nearest([7.0, 1e9], kv.E2M1).tolist() == [7, 7]


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_quantiser_blocks_round_trip(d, page):
    x = np.random.default_rng(0).normal(size=(page, d))
    x[3] = 0
    code, s8 = kv.quantise(x, 0.5)
    c2, s2 = kv.unblock(kv.block(code, s8), page, d)
    assert np.array_equal(code, c2) and np.array_equal(s8, s2)
    y = kv.dequantise(code, s8, 0.5)
    # half a step of the coarsest code spacing (2 of 6) plus the scale's own rounding, 2^-4
    top = np.abs(x).reshape(page, -1, 16).max(-1).repeat(16, -1)
    assert (np.abs(y - x) <= top * (1 / 6 + 2 ** -4) + 0.5 * 2 ** -9).all()
    assert (y[3] == 0).all()
    x[5, 7] = np.inf
    assert np.isnan(kv.dequantise(*kv.quantise(x))[5]).all()


def test_cached_values_fit_bf16():
    v = np.outer(kv.E2M1, kv.E4M3).reshape(-1)
    assert np.array_equal(torch.tensor(v).bfloat16().double().numpy(), v)
    assert np.array_equal(torch.tensor(v).half().double().numpy(), v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_pairs_and_its_inverse_is_the_gradient(interleaved):
    turns, _ = ea.rope_turns(32, device="cpu")
    turns = turns.tolist()
    rng = np.random.default_rng(1)
    x, pos = rng.normal(size=(5, 64)), [0, 1, 77, 100000, -3]
    y = kv.rope(x, pos, turns, interleaved, mscale=1.5)
    assert np.array_equal(y[:, 32:], x[:, 32:])
    assert np.allclose(y[0, :32], 1.5 * x[0, :32], rtol=1e-15)
    f = [10000.0 ** (-2 * i / 32) for i in range(16)]
    a, b = (4, 5) if interleaved else (2, 18)
    z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * np.array(pos) * f[2]) * 1.5
    # the table's step is off by 2^-53 of itself at most (a double), times positions up to 1e5
    assert np.allclose(y[:, a] + 1j * y[:, b], z, rtol=0, atol=1e-10)
    # gradient of sum(w y) by differences against the inverse map on w
    w = rng.normal(size=x.shape)
    g = kv.rope(w, pos, turns, interleaved, inverse=True, mscale=1.5)
    for n, i in ((1, 0), (2, 17), (3, 31), (4, 40)):
        step = np.zeros_like(x)
        step[n, i] = 1e-3
        diff = (w * (kv.rope(x + step, pos, turns, interleaved, mscale=1.5)
                     - kv.rope(x - step, pos, turns, interleaved, mscale=1.5))).sum() / 2e-3
        # the map is linear: only the rounding of the differences is left
        want = g[n, i]
        assert abs(diff - want) < 1e-9


def test_rope_tables():
    plain, one = ea.rope_turns(128, device="cpu")
    assert plain.dtype == torch.int64 and one == 1.0
    unit = 2 * math.pi / 2.0 ** 64
    assert math.isclose(int(plain[0]) * unit, 1.0, rel_tol=1e-15)
    lin, _ = ea.rope_turns(128, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(lin.double() * 4, plain.double(), rtol=1e-12)
    base, _ = ea.rope_turns(128, scaling="base", factor=4.0, device="cpu")
    assert base[0] == plain[0] and math.isclose(int(base[-1]) * 4, int(plain[-1]), rel_tol=1e-12)
    parts, m = ea.rope_turns(128, scaling="parts", factor=4.0, context=4096, device="cpu")
    assert parts[0] == plain[0] and math.isclose(int(parts[-1]) * 4, int(plain[-1]), rel_tol=1e-12)
    ratio = (parts.double() / plain.double()).numpy()
    assert (np.diff(ratio) <= 1e-12).all() and math.isclose(m, 1 + 0.1 * math.log(4))
    for bad in (dict(scaling="other"), dict(factor=0.5), dict(base=float("nan"))):
        with pytest.raises(ValueError):
            ea.rope_turns(128, device="cpu", **bad)
    with pytest.raises(ValueError):
        ea.rope_turns(7, device="cpu")


def test_page_plan_hands_out_each_page_once():
    rng = np.random.default_rng(2)
    page, width, B = 16, 6, 9
    table = np.arange(B * width).reshape(B, width)
    lens = rng.integers(0, 80, B).tolist()
    used = sum(math.ceil(n / page) for n in lens)
    free = [int(p) for b in range(B) for p in table[b, math.ceil(lens[b] / page):]]
    queue, state = free + [-5] * used, [0, len(free)]
    tab = table.tolist()
    for _ in range(40):
        new = rng.integers(-1, 20, B).tolist()
        lens, off, pos, slots, state, tab, queue = kv.page_plan(lens, new, tab, queue, state, page, 200)
        held = [p for b in range(B) for p in tab[b][:math.ceil(lens[b] / page)]]
        idle = [queue[(state[0] + i) % len(queue)] for i in range(state[1])]
        assert sorted(held + idle) == list(range(B * width))
        real = [s for s in slots if s >= 0]
        assert len(set(real)) == len(real)


def test_attention_matches_softmax():
    rng = np.random.default_rng(3)
    d, page, Hkv, Hq = 64, 16, 2, 4
    x = rng.normal(size=(2, Hkv, 2, page, d))
    cache = np.stack([[[kv.block(*kv.quantise(x[p, h, n])) for n in range(2)] for h in range(Hkv)]
                      for p in range(2)])
    y = np.stack([[[kv.dequantise(*kv.quantise(x[p, h, n])) for n in range(2)] for h in range(Hkv)]
                  for p in range(2)])
    q = rng.normal(size=(3, Hq, d))
    table = np.array([[1, 0]])
    o, lse, *_ = kv.kv4_attention(q, cache, table, [20], [0, 3], d, 0.3, True)
    k = torch.tensor(np.concatenate([y[1, :, 0], y[0, :, 0, :4]], 1)).repeat_interleave(2, 0)
    v = torch.tensor(np.concatenate([y[1, :, 1], y[0, :, 1, :4]], 1)).repeat_interleave(2, 0)
    s = 0.3 * torch.tensor(q).transpose(0, 1) @ k.transpose(1, 2)
    s = s.masked_fill(torch.ones(3, 20).triu(18).bool(), -math.inf)
    assert np.allclose(o, (s.softmax(-1) @ v).transpose(0, 1), atol=1e-12)
    assert np.allclose(lse, s.logsumexp(-1).T, atol=1e-12)
    o, lse, *_ = kv.kv4_attention(q, cache, table, [2], [0, 3], d, 0.3, True)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1:]).all()


def test_page_plan_of_a_ring_too_small_gives_no_page_twice():
    """1 takes two pages while 0 gives two back to a full ring: those are lost, 1's stay its own."""
    out = kv.page_plan([32, 0], [-1, 32], [[10, 11], [0, 0]], [1, 2, 3, 4], [0, 4], 16, 32)
    assert out[4] == [2, 2] and out[5][1] == [1, 2] and out[6] == [1, 2, 3, 4]


def _pi_times(scale):
    """floor(pi * scale), nearly: 16 atan(1/5) - 4 atan(1/239) in integers, with guard digits."""
    guard = 10 ** 20

    def atan_inverse(n):
        term, total, k = scale * guard // n, 0, 0
        while term:
            total += (-term if k % 2 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total

    return (16 * atan_inverse(5) - 4 * atan_inverse(239)) // guard


def _root(x, n, one):
    """The n-th root of x / one in units of 1 / one, by bisection in integers."""
    lo, hi = 0, max(x, one) + 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        y = one
        for _ in range(n):
            y = y * mid // one
        lo, hi = (mid, hi) if y <= x else (lo, mid)
    return lo


@pytest.mark.parametrize("r,base", [(128, 10000), (64, 500000), (16, 10000), (48, 10007)])
@pytest.mark.parametrize("scaling,factor", [(None, 1), ("linear", 4), ("base", 8)])
def test_rope_turns_are_right_to_their_last_bit(r, base, scaling, factor):
    """Against roots and pi in integers of 60 digits: entries are the rounded f_i / (2 pi), so off by half a
    unit of 2^-64 turn at most (and 2^-40 of one for the integers here)."""
    one = 10 ** 60
    turns = ea.rope_turns(r, base=base, scaling=scaling, factor=factor, device="cpu")[0].tolist()
    ratio = one * one // _root(base * one, r // 2, one)  # f_1 / f_0 of the plain table
    if scaling == "base":  # (base * factor^(r / (r - 2)))^(-2 / r) = base^(-2 / r) factor^(-2 / (r - 2))
        ratio = ratio * one // _root(factor * one, (r - 2) // 2, one)
    f, two_pi = one // (factor if scaling == "linear" else 1), 2 * _pi_times(one)
    for t in turns:
        units = f * one // two_pi * 2 ** 64
        assert abs(t * one - units) <= one // 2 + one // 2 ** 40
        f = f * ratio // one


def test_rope_turns_by_parts_and_under_a_callers_decimal_context():
    """Each entry by parts is the mean, with the ramp's weight, of the plain one and of the one divided by
    the factor: three roundings.  The caller's precision is neither used nor changed."""
    import decimal

    with decimal.localcontext() as ctx:
        ctx.prec = 3
        plain = ea.rope_turns(128, device="cpu")[0].tolist()
        parts = ea.rope_turns(128, scaling="parts", factor=8.0, context=4096, device="cpu")[0].tolist()
        assert decimal.getcontext().prec == 3
    assert plain == ea.rope_turns(128, device="cpu")[0].tolist()
    at = lambda times: 128 * math.log(4096 / (times * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = math.floor(at(32.0)), math.ceil(at(1.0))
    for i, (x, y) in enumerate(zip(plain, parts)):
        w = min(max(i - lo, 0), hi - lo)  # of hi - lo
        assert abs(8 * (hi - lo) * y - x * (w + 8 * (hi - lo - w))) <= 8 * (hi - lo)
