"""Rotary positions on the GPU against the fp64 reference, element by element."""
import math

import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import kv

pytestmark = pytest.mark.gpu


def numpy64(t):
    return t.double().cpu().numpy()


def check(got, x, positions, turns, mscale=1.0, **kw):
    """|y - y64| <= half a bf16 step of y64, plus fp32's part: the angle (2^-25 half turns, 2^-23.3
    radians), two units in the last place of the cosine and its product with mscale (2^-22.7) and
    the products and their sum (2^-23.4), each times |a| + |b| <= sqrt(2) hypot(a, b): below 2^-20
    mscale hypot(a, b)."""
    r = 2 * len(turns)
    want = kv.rope(x, positions, turns, mscale=mscale, **kw)
    il = kw.get("interleaved", False)
    first = slice(0, r, 2) if il else slice(0, r // 2)
    second = slice(1, r, 2) if il else slice(r // 2, r)
    size = np.zeros_like(want)
    size[..., first] = size[..., second] = np.hypot(x[..., first], x[..., second])
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * abs(mscale) * size
    assert (np.abs(numpy64(got) - want) <= tol).all()
    assert np.array_equal(numpy64(got)[..., r:], x[..., r:])


def draws(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 16), (128, 128), (128, 48)])
def test_packed_tokens(d, r, interleaved, inverse):
    turns, m = ea.rope_turns(r, scaling="parts", factor=4.0)
    T = 13
    q, k = draws(T, 5, d), draws(T, 2, d, seed=1)
    pos = torch.tensor([0, 1, 2, 3, 1000, 131071, 1 << 20, (1 << 31) - 1, -1, -5, 7, 7, 99999],
                       dtype=torch.int32).cuda()
    qo, ko = ea.rope(q, k, pos, turns, interleaved=interleaved, inverse=inverse, mscale=m)
    for x, y in ((q, qo), (k, ko)):
        check(y.transpose(0, 1), numpy64(x).swapaxes(0, 1), pos.tolist(), turns.tolist(), m,
              interleaved=interleaved, inverse=inverse)


@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (2, 3, 130), (1, 9, 1000)])
@pytest.mark.parametrize("per_batch", [False, True])
def test_dense_heads(B, H, N, per_batch):
    turns, _ = ea.rope_turns(128)
    q, k = draws(B, H, N, 128), draws(B, 1, N, 128, seed=2)
    pos = torch.arange(N, dtype=torch.int32)
    if per_batch:
        pos = torch.stack([pos + 1000 * b for b in range(B)])
    qo, ko = ea.rope(q, k, pos.cuda(), turns)
    for b in range(B):
        p = (pos[b] if per_batch else pos).tolist()
        check(qo[b], numpy64(q[b]), p, turns.tolist())
        check(ko[b], numpy64(k[b]), p, turns.tolist())


def test_strided_slices_in_place_and_one_tensor():
    """q and k as slices of one projection row, rotated in place; the values beside them stay."""
    turns, _ = ea.rope_turns(64)
    T, row = 37, draws(37, 4 + 2 + 2, 64)
    before = row.clone()
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32, generator=torch.Generator().manual_seed(3)).cuda()
    q, k = row[:, :4], row[:, 4:6]
    want_q, want_k = ea.rope(before[:, :4], before[:, 4:6], pos, turns)
    got = ea.rope(q, k, pos, turns, q_out=q, k_out=k)
    assert got[0].data_ptr() == row.data_ptr()
    assert torch.equal(row[:, :4], want_q) and torch.equal(row[:, 4:6], want_k)
    assert torch.equal(row[:, 6:], before[:, 6:])
    alone, none = ea.rope(before[:, :4], None, pos, turns)
    assert none is None and torch.equal(alone, want_q)
    # [B, H, N, d] seen through a transpose (rows of a head far apart)
    x = draws(2, 50, 3, 64)
    pos = torch.arange(50, dtype=torch.int32).cuda()
    y, _ = ea.rope(x.transpose(1, 2), None, pos, turns)
    z, _ = ea.rope(x.transpose(1, 2).contiguous(), None, pos, turns)
    assert torch.equal(y, z)


def test_infinities_and_nan_stay_in_their_pair():
    turns, _ = ea.rope_turns(128)
    x = draws(3, 2, 128)
    y0, _ = ea.rope(x, None, torch.arange(3, dtype=torch.int32).cuda(), turns)
    x[1, 1, 5], x[2, 0, 70] = math.nan, math.inf
    y, _ = ea.rope(x, None, torch.arange(3, dtype=torch.int32).cuda(), turns)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[1, 1, [5, 69]] = touched[2, 0, [6, 70]] = True
    assert torch.equal(torch.isfinite(y), ~touched)
    assert torch.equal(y[~touched], y0[~touched])


def test_gradient_by_differences():
    """L = sum w . rope(x): the inverse map on w against differences of the (linear) kernel.  With a
    step of 64 a pair's two outputs are at most m (64.25 + |x|) < 70 m, each rounded by 2^-8 of that in
    both calls: 4 roundings, times |w| <= 4, over a difference of 128 in x (64 here, for room).  The
    inverse itself is off by 2^-8 |g|."""
    turns, m = ea.rope_turns(64, scaling="parts", factor=8.0)
    x, w = draws(4, 1, 64), draws(4, 1, 64, seed=1).clamp(-4, 4)
    pos = torch.tensor([3, 500, 40000, 999999], dtype=torch.int32).cuda()
    g, _ = ea.rope(w, None, pos, turns, inverse=True, mscale=m)
    f = lambda z: (w.double() * ea.rope(z, None, pos, turns, mscale=m)[0].double()).sum((1, 2))  # noqa: E731
    for i in (0, 9, 31, 32, 63):
        step = torch.zeros_like(x)
        step[..., i] = 64.0
        up, down = (x + step), (x - step)
        h = (up.double() - down.double())[..., i].squeeze(1)  # the step that bf16 made of it
        diff = (f(up) - f(down)) / h
        tol = 4 * 4 * 2.0 ** -8 * m * 70 / 64 + 2.0 ** -8 * g[..., i].abs().double().squeeze(1)
        assert ((diff - g[..., i].double().squeeze(1)).abs() <= tol).all()


def test_refusals():
    turns, _ = ea.rope_turns(128)
    q, pos = draws(4, 2, 128), torch.arange(4, dtype=torch.int32).cuda()
    for args in ((q.float(), None, pos, turns), (q, None, pos.long(), turns), (q, None, pos[:3], turns),
                 (q, draws(5, 2, 128), pos, turns), (q, draws(4, 2, 64), pos, turns),
                 (q, None, pos, turns.int()), (q.transpose(1, 2), None, pos, turns),
                 (q, None, pos.cpu(), turns), (q, None, pos, turns.cpu())):
        with pytest.raises(ValueError):
            ea.rope(*args)
    with pytest.raises(ea.AttentionError):
        ea.rope(draws(4, 2, 64), None, pos, turns)  # more rotated values than the head has
    with pytest.raises(ea.AttentionError):
        ea.rope(draws(5, 2, 132)[1:, :, 4:], None, pos, turns)  # strides of 132


def test_training_step_gradients():
    """rope -> fwd -> bwd -> rope inverse against fp64 autograd of the same chain.  The attention
    backward's gate is 1e-2 of max |g| per tensor; rotating back adds half a bf16 step of a pair
    (2^-8 * sqrt 2) to it, and the forward rounding of q and k (2^-8 each) moves scores by about
    2^-8 * |s|, which moves P, and so the gradients, by about 2^-7 relative: 4e-2 in all."""
    B, H, N, d = 1, 2, 200, 128
    turns, _ = ea.rope_turns(d)
    pos = torch.arange(N, dtype=torch.int32).cuda()
    q, k, v, do = (draws(B, H, N, d, seed=s) for s in range(4))
    qr, kr = ea.rope(q, k, pos, turns)
    o, lse = ea.fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = ea.bwd(qr, kr, v, o, lse, do, causal=True)
    dq, dk = ea.rope(dqr, dkr, pos, turns, inverse=True)
    f = torch.tensor([10000.0 ** (-2 * i / d) for i in range(d // 2)], dtype=torch.float64).cuda()
    angle = pos.double()[:, None] * f

    def turn(x):
        a, b = x[..., :d // 2], x[..., d // 2:]
        c, s = angle.cos(), angle.sin()
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    s = turn(leaves[0]) @ turn(leaves[1]).transpose(-1, -2) / math.sqrt(d)
    s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -math.inf)
    ((s.softmax(-1) @ leaves[2]) * do.double()).sum().backward()
    for got, leaf in zip((dq, dk, dv), leaves):
        assert (got.double() - leaf.grad).abs().max() <= 4e-2 * leaf.grad.abs().max()
