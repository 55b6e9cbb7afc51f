"""The fp64 reference of trees of drafted tokens and of rotary positions with several axes, pinned by small
examples worked by hand and by a chain, which is the causal mask (CPU only)."""
import numpy as np
import pytest
import torch

import exact_attention_13_gb300 as ea
from oracle import kv, tree


def test_plan_by_hand():
    #        0          request 1: 0 -> 1, and 2 on the cached token
    #      1   2
    #     3 4   5
    parents = [-1, 0, 0, 1, 1, 2] + [-1, 0, -1]
    pos, seen = tree.tree_plan(parents, [0, 6, 9], [10, 3], 1)
    assert pos.tolist() == [10, 11, 11, 12, 12, 12, 3, 4, 3]
    assert [np.flatnonzero(r).tolist() for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [0, 2, 5],
                                                         [0], [0, 1], [2]]
    assert tree.bits(seen)[:, 0].tolist() == [1, 3, 5, 11, 19, 37, 1, 3, 4]
    high = np.zeros((1, 64), dtype=bool)
    high[0, 31] = high[0, 32] = True
    assert tree.bits(high).tolist() == [[-2 ** 31, 1]]


def test_accept_by_hand():
    parents = [-1, 0, 0, 1, 1, 2] + [-1, 0, 1] + [-1, 0]
    tokens = [9, 5, 6, 7, 7, 8] + [4, 3, 2] + [1, 1]
    choices = [5, 7, 8, 50, 51, 52] + [2, 60, 61] + [1, 1]
    table = np.arange(12).reshape(3, 4)
    slots = [10 + i for i in range(6)] + [100, 101, 102] + [-1, -1]
    got = tree.tree_accept(parents, tokens, choices, [30, 14, 5], [36, 17, 5], [0, 6, 9, 11], slots,
                           table, [77] * 6, [4, 1], 16, 1)
    # request 0: 0, its child 1 (token 5), of 3 and 4 (both 7) the first; 1: node 0 alone; 2: refused
    assert got[0] == [33, 15, 5] and got[1] == [3, 1, 0]
    assert got[2] == [0, 1, 3, -1, -1, -1, 0, -1, -1, -1, -1] and got[3] == [50, 2, -1]
    assert got[4] == [10, 11, 13, -1, -1, -1, 100, -1, -1, -1, -1]
    # request 0 holds 3 pages for 36 tokens and for 33; request 1 two for 17 and one for 15
    assert got[5] == [4, 2] and got[6] == [77, 77, 77, 77, 77, 5]


def test_move_by_hand():
    cache = np.arange(2 * 1 * 2 * 16 * 36, dtype=np.int64).reshape(2, 1, 2, 16 * 36)
    got = tree.kv4_move(cache, [3, 20, -1, 5], [0, 1, 2, 40], [0, 4], [4], 64)
    for src, dst in ((3, (0, 0)), (20, (0, 1))):
        p, r = divmod(src, 16)
        assert np.array_equal(got[dst[0], :, :, dst[1] * 32:dst[1] * 32 + 32], cache[p, :, :, r * 32:r * 32 + 32])
        assert np.array_equal(got[0, :, :, 512 + dst[1] * 4:516 + dst[1] * 4], cache[p, :, :, 512 + r * 4:516 + r * 4])
    assert (got != cache).sum() == 2 * 2 * 36


def test_a_chain_is_the_causal_mask():
    rng = np.random.default_rng(0)
    d, page, lens, nodes = 64, 16, [37, 3, 0], [5, 4, 2]
    cache = rng.integers(0, 120, (12, 2, 2, page * 36)).astype(np.uint8)
    table = rng.permutation(12).reshape(3, 4)
    off = [0, 5, 9, 11]
    parents = [i - 1 for n in nodes for i in range(n)]
    _, seen = tree.tree_plan(parents, off, [0] * 3, 1)
    q = rng.standard_normal((11, 4, d))
    a = tree.kv4_tree_attention(q, cache, table, lens, off, seen, d, 0.1)
    b = kv.kv4_attention(q, cache, table, lens, off, d, 0.1, True)
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-12, atol=1e-12, equal_nan=True)


def test_axes_of_one_position_are_rope():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((3, 5, 64)), [0, 1, 77, 2 ** 31 - 1, -4]
    turns = [int(t) for t in rng.integers(1, 2 ** 62, 24)]
    axes = rng.integers(0, 3, 24)
    for kw in ({}, dict(interleaved=True), dict(inverse=True, mscale=1.5)):
        assert np.allclose(tree.rope_axes(x, [pos] * 3, turns, axes, **kw), kv.rope(x, pos, turns, **kw),
                           rtol=0, atol=1e-12)


def test_axis_pairs():
    pairs = lambda *a, **kw: ea.rope_axis_pairs(*a, device="cpu", **kw).tolist()  # noqa: E731
    assert pairs((2, 3, 3)) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert pairs((4, 2, 2), cycled=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert pairs((2, 0, 1), cycled=True) == [0, 2, 0]
    assert pairs((5,)) == [0] * 5
    for bad in ((), (1, 2, 3, 4, 5), (-1, 4), (0, 0), (40, 30)):
        with pytest.raises(ValueError):
            pairs(bad)
    assert ea.rope_axis_pairs((16, 24, 24), device="cpu").dtype is torch.uint8
