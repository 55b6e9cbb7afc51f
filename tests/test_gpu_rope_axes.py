"""Rotary positions with several axes on the GPU against the fp64 reference, element by element."""
import math

import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import tree

pytestmark = pytest.mark.gpu


def numpy64(t):
    return t.double().cpu().numpy()


def draws(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def places(A, *shape, top=5000, seed=3):
    return torch.randint(0, top, (A, *shape), dtype=torch.int32, generator=torch.Generator().manual_seed(seed)).cuda()


def check(got, x, positions, turns, axes, mscale=1.0, **kw):
    """Half a bf16 step of the result (2^-8 relative is a whole one) and fp32's part: the angle (2^-25 half
    turns, 2^-23.3 radians), two units in the last place of the cosine and its product with mscale (2^-22.7), the
    products and their sum (2^-23.4), each times |a| + |b| <= sqrt(2) hypot(a, b): below 2^-20 mscale hypot(a, b)."""
    r = 2 * len(turns)
    want = tree.rope_axes(x, positions, turns, axes, mscale=mscale, **kw)
    il = kw.get("interleaved", False)
    first = slice(0, r, 2) if il else slice(0, r // 2)
    second = slice(1, r, 2) if il else slice(r // 2, r)
    size = np.zeros_like(want)
    size[..., first] = size[..., second] = np.hypot(x[..., first], x[..., second])
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * abs(mscale) * size
    assert (np.abs(numpy64(got) - want) <= tol).all()
    assert np.array_equal(numpy64(got)[..., r:], x[..., r:])


SECTIONS = {16: (2, 3, 3), 32: (8, 8), 48: (24,), 64: (8, 12, 12), 128: (16, 24, 24), 96: (12, 12, 12, 12)}


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved,cycled", [(False, False), (True, True)])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 16), (64, 32), (128, 128), (128, 48), (128, 96)])
def test_packed_tokens(d, r, interleaved, cycled, inverse):
    turns, m = ea.rope_turns(r, scaling="parts", factor=4.0)
    axes = ea.rope_axis_pairs(SECTIONS[r], cycled=cycled)
    T, A = 13, len(SECTIONS[r])
    q, k = draws(T, 5, d), draws(T, 2, d, seed=1)
    pos = places(A, T, top=1 << 20)
    pos[:, :8] = torch.tensor([0, 1, -1, 131071, (1 << 31) - 1, -(1 << 31), 7, 99999], dtype=torch.int32).cuda()
    pos[-1, :8] += 1
    qo, ko = ea.rope_axes(q, k, pos, turns, axes, interleaved=interleaved, inverse=inverse, mscale=m)
    for x, y in ((q, qo), (k, ko)):
        check(y.transpose(0, 1), numpy64(x).swapaxes(0, 1), pos.tolist(), turns.tolist(), axes.tolist(), m,
              interleaved=interleaved, inverse=inverse)


@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (2, 3, 130), (1, 9, 1000)])
@pytest.mark.parametrize("per_batch", [False, True])
def test_dense_heads(B, H, N, per_batch):
    turns, _ = ea.rope_turns(128)
    axes = ea.rope_axis_pairs((16, 24, 24))
    q, k = draws(B, H, N, 128), draws(B, 1, N, 128, seed=2)
    pos = places(3, B, N) if per_batch else places(3, N)
    qo, ko = ea.rope_axes(q, k, pos, turns, axes)
    for b in range(B):
        p = (pos[:, b] if per_batch else pos).tolist()
        check(qo[b], numpy64(q[b]), p, turns.tolist(), axes.tolist())
        check(ko[b], numpy64(k[b]), p, turns.tolist(), axes.tolist())


def test_equal_positions_are_one_axis():
    """Text tokens: the same bits as ``rope``; so with an axis that there is not, which counts as the first."""
    turns, _ = ea.rope_turns(128)
    q, k = draws(50, 6, 128), draws(50, 2, 128, seed=1)
    pos = places(1, 50, top=100000)
    want = ea.rope(q, k, pos[0], turns)
    for axes in (ea.rope_axis_pairs((16, 24, 24)), ea.rope_axis_pairs((20, 22, 22), cycled=True)):
        got = ea.rope_axes(q, k, pos.expand(3, -1).contiguous(), turns, axes)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for other in (1, 3, 4, 200, 255):
        axes = torch.full((64,), other, dtype=torch.uint8).cuda()
        got = ea.rope_axes(q, k, pos, turns, axes)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_strided_slices_in_place_one_tensor_and_other_streams():
    turns, _ = ea.rope_turns(64)
    axes = ea.rope_axis_pairs((8, 12, 12))
    T, row = 37, draws(37, 4 + 2 + 2, 64)
    before = row.clone()
    pos = places(3, T)
    q, k = row[:, :4], row[:, 4:6]
    want_q, want_k = ea.rope_axes(before[:, :4], before[:, 4:6], pos, turns, axes)
    got = ea.rope_axes(q, k, pos, turns, axes, q_out=q, k_out=k)
    assert got[0].data_ptr() == row.data_ptr()
    assert torch.equal(row[:, :4], want_q) and torch.equal(row[:, 4:6], want_k)
    assert torch.equal(row[:, 6:], before[:, 6:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alone, none = ea.rope_axes(before[:, :4], None, pos, turns, axes)
    torch.cuda.current_stream().wait_stream(side)
    assert none is None and torch.equal(alone, want_q)
    empty = ea.rope_axes(before[:0, :4], before[:0, 4:6], pos[:, :0].contiguous(), turns, axes)
    assert empty[0].shape == (0, 4, 64)


def test_gradient_is_the_transpose():
    """<rope(x), g> = <x, inverse(g)> for the linear map, and differences of a loss along a direction: every
    value is off by 2^-8 relative at most on each side (the roundings of both results), so the sums are by
    2^-8 times the sums of the absolute products, and a difference likewise."""
    turns, _ = ea.rope_turns(128)
    axes = ea.rope_axis_pairs((16, 24, 24), cycled=True)
    x, g, e = draws(2, 4, 70, 128), draws(2, 4, 70, 128, seed=5), draws(2, 4, 70, 128, seed=6)
    pos = places(3, 2, 70)
    y, _ = ea.rope_axes(x, None, pos, turns, axes, mscale=1.25)
    dx, _ = ea.rope_axes(g, None, pos, turns, axes, inverse=True, mscale=1.25)
    left, right = numpy64(y) * numpy64(g), numpy64(x) * numpy64(dx)
    assert abs(left.sum() - right.sum()) <= 2.0 ** -8 * (np.abs(left).sum() + np.abs(right).sum())
    up, _ = ea.rope_axes((x + e).bfloat16(), None, pos, turns, axes, mscale=1.25)
    step = numpy64((x + e).bfloat16()) - numpy64(x)
    diff, slope = (numpy64(up) - numpy64(y)) * numpy64(g), step * numpy64(dx)
    room = 2.0 ** -8 * ((np.abs(numpy64(up)) + np.abs(numpy64(y))) * np.abs(numpy64(g))).sum()
    assert abs(diff.sum() - slope.sum()) <= room + 2.0 ** -8 * np.abs(slope).sum()


def test_training_step_with_attention():
    """rope_axes -> fwd -> bwd -> inverse, with the gradients of the rotated tensors turned back, and the same
    step captured into a graph: the same bits."""
    turns, _ = ea.rope_turns(64)
    axes = ea.rope_axis_pairs((8, 12, 12))
    q, k, v, do = (draws(1, 2, 160, 64, seed=s) for s in range(4))
    pos = places(3, 160)

    def step():
        qr, kr = ea.rope_axes(q, k, pos, turns, axes)
        o, lse = ea.fwd(qr, kr, v, causal=True)
        dqr, dkr, dv = ea.bwd(qr, kr, v, o, lse, do, causal=True)
        dq, dk = ea.rope_axes(dqr, dkr, pos, turns, axes, inverse=True)
        return o, dqr, dq, dk, dv

    want = step()
    check(want[2][0], numpy64(want[1][0]), pos.tolist(), turns.tolist(), axes.tolist(), inverse=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_refusals():
    q, k = draws(8, 4, 128), draws(8, 2, 128)
    turns, _ = ea.rope_turns(128)
    axes, pos = ea.rope_axis_pairs((16, 24, 24)), places(3, 8)
    ea.rope_axes(q, k, pos, turns, axes)
    bad = [dict(positions=pos[0]), dict(positions=places(5, 8)), dict(positions=pos.long()),
           dict(positions=places(3, 9)), dict(positions=places(3, 16)[:, ::2]), dict(positions=pos.cpu()),
           dict(axes=axes[:32]), dict(axes=axes.int()), dict(axes=axes.cpu()), dict(turns=turns[:32]),
           dict(k=k[:7]), dict(k=k.float()), dict(q=q.cpu())]
    for change in bad:
        args = dict(q=q, k=k, positions=pos, turns=turns, axes=axes) | change
        with pytest.raises(ValueError):
            ea.rope_axes(**args)
    with pytest.raises(ea.AttentionError):  # four bytes off the alignment of the axes
        ea.rope_axes(q, k, pos, turns, torch.zeros(72, dtype=torch.uint8).cuda()[4:68])
    with pytest.raises(ea.AttentionError):
        ea.rope_axes(q, k, pos, turns, axes, mscale=math.inf)
