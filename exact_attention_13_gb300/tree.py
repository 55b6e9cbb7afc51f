"""Trees of drafted tokens over the paged 4-bit cache: their plan, attention, what is accepted of them, and
the accepted rows' way to their places.  Like kv.py these functions check and marshal arguments only.

A request's new tokens are the nodes of a tree: node 0 is the token that the step before chose, every other
one a draft that hangs on an earlier node of its request (``parents``: its number among them; -1: on the
last cached token).  A step that checks all of them at once, every length on the device:

    plan = ea.page_plan(lens, nodes, table, queue, queue_state, page_size=64, num_tokens=T)
    tree = ea.tree_plan(parents, plan.q_offsets, lens, max_nodes=64)
    q, k = ea.rope(q, k, tree.positions, turns)                       # for each layer:
    ea.kv4_append(k, v, cache, plan.slots)
    o, lse = ea.kv4_tree_fwd(q, cache, table, plan.lens, plan.q_offsets, tree.seen, max_q=...)
    # the model's choice at each node: choices [T]; caches: a list, one of each layer
    got = ea.tree_accept(parents, tree.seen, tokens, choices, lens, plan.lens, plan.q_offsets, plan.slots,
                         table, queue, plan.queue_state, page_size=64)
    ea.kv4_move(caches, got.sources, plan.slots, plan.q_offsets, got.counts, d)   # all layers at once
    lens, queue_state = got.lens, got.queue_state                     # got.next_tokens: the next roots
"""
from __future__ import annotations

import array
import functools
import math
from typing import NamedTuple

import torch

from .kv import _bf16, _cache_shape, _f32, _fn, _i32, _ints, _most, _run

_most_nodes = 256  # nodes of a request that others can see


class TreePlan(NamedTuple):
    """What ``tree_plan`` wrote (int32 CUDA tensors)."""

    positions: torch.Tensor    # [T] cached tokens of the request + depth of the node
    seen: torch.Tensor         # [T, ceil(max_nodes / 32)] bit i: node i lies on the node's way up


class TreeAccept(NamedTuple):
    """What ``tree_accept`` wrote (int32 CUDA tensors)."""

    lens: torch.Tensor         # [B] lengths after the step
    counts: torch.Tensor       # [B] accepted nodes
    path: torch.Tensor         # [T] accepted nodes of each request from its first row on, -1 behind them
    next_tokens: torch.Tensor  # [B] the choice behind the last accepted node (-1: none accepted)
    sources: torch.Tensor      # [T] slots of the nodes of `path`
    queue_state: torch.Tensor  # [2] head and count of the free pages after the step


def tree_plan(parents, q_offsets, lens, max_nodes: int, out: TreePlan | None = None) -> TreePlan:
    """Positions and masks of trees of drafted tokens (one launch).

    ``parents`` int32 [T]: each node's parent, a smaller number among its request's nodes, or -1 (any other
    value counts as -1); ``q_offsets`` int32 [B + 1]: first node of each request; ``lens`` int32 [B]: cached
    tokens before the step.  ``max_nodes`` (1 to 256) is rounded up to a multiple of 32: that many nodes of a
    request have a bit, nodes past them are seen by none, themselves included, and are not accepted.  It makes
    room for the nodes there are; to check fewer of them, bring fewer.  Rows past the last request get position 0
    and no bits."""
    index = parents.get_device()
    if index < 0 or parents.dim() != 1 or lens.dim() != 1 or not 1 <= max_nodes <= _most_nodes:
        raise ValueError("parents and lens must be int32 CUDA vectors, max_nodes in [1, 256]")
    T, B, words = parents.shape[0], lens.shape[0], (max_nodes + 31) // 32
    _ints(parents, (T,), index, "parents")
    _ints(q_offsets, (B + 1,), index, "q_offsets")
    _ints(lens, (B,), index, "lens")
    if out is None:
        out = TreePlan(torch.empty(T, dtype=_i32, device=parents.device),
                       torch.empty((T, words), dtype=_i32, device=parents.device))
    else:
        _ints(out[0], (T,), index, "out.positions")
        _ints(out[1], (T, words), index, "out.seen")
    if T == 0:
        return out
    _run("fa_tree_plan", index, parents.data_ptr(), q_offsets.data_ptr(), lens.data_ptr(), B, T, words,
         out[0].data_ptr(), out[1].data_ptr())
    return out


def _seen(seen, T, index):
    if seen.dim() != 2 or not 1 <= seen.shape[1] <= _most_nodes // 32:
        raise ValueError("seen must be [T, words] as tree_plan makes it")
    _ints(seen, (T, seen.shape[1]), index, "seen")
    return seen.shape[1]


def tree_accept(parents, seen, tokens, choices, lens, new_lens, q_offsets, slots, table, queue, queue_state,
                page_size: int, out: TreeAccept | None = None) -> TreeAccept:
    """What a step accepts of its trees (one launch for up to 64 requests, else two).

    ``tokens`` int32 [T]: the token at each node; ``choices`` int32 [T]: the token that the model chose behind
    it (greedy or drawn).  Node 0 of a request is accepted, and so is every child of an accepted node that holds
    its parent's choice (of several the first).  ``parents`` and ``seen``: as for and from ``tree_plan``;
    ``lens``, ``new_lens``: lengths before the step and with the nodes (``page_plan``'s inputs and outputs; a
    request without growth was refused or had ended: nothing is accepted); ``slots`` [T]: the nodes' slots.
    Pages behind the last one that a new length needs go back to the ring ``queue`` (in place), behind the free
    ones that ``queue_state`` says.  All int32.  ``out``: results to write into; none may be an input."""
    index = parents.get_device()
    if (index < 0 or parents.dim() != 1 or lens.dim() != 1 or table.dim() != 2 or queue.dim() != 1
            or not 0 < page_size <= _most):
        raise ValueError("parents, lens and queue must be int32 CUDA vectors, table [B, width]")
    T, B, width, cap = parents.shape[0], lens.shape[0], table.shape[1], queue.shape[0]
    words = _seen(seen, T, index)
    for t, shape, name in ((parents, (T,), "parents"), (tokens, (T,), "tokens"), (choices, (T,), "choices"),
                           (slots, (T,), "slots"), (lens, (B,), "lens"), (new_lens, (B,), "new_lens"),
                           (q_offsets, (B + 1,), "q_offsets"), (table, (B, width), "table"),
                           (queue, (cap,), "queue"), (queue_state, (2,), "queue_state")):
        _ints(t, shape, index, name)
    sizes = (B, B, T, B, T, 2)
    if out is None:
        # one allocation for the six parts, as in page_plan
        flat = torch.empty(3 * B + 2 * T + 2, dtype=_i32, device=parents.device)
        out = TreeAccept._make(torch.unsafe_split_with_sizes(flat, sizes))
    else:
        for t, n, name in zip(out, sizes, TreeAccept._fields):
            _ints(t, (n,), index, f"out.{name}")
    if B == 0:
        raise ValueError("there are no requests")
    _run("fa_tree_accept", index, parents.data_ptr(), seen.data_ptr(), words, tokens.data_ptr(),
         choices.data_ptr(), lens.data_ptr(), new_lens.data_ptr(), q_offsets.data_ptr(), slots.data_ptr(),
         table.data_ptr(), width, queue.data_ptr(), cap, queue_state.data_ptr(), B, page_size, T,
         out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(),
         out[5].data_ptr())
    return out


def kv4_move(caches, sources, slots, q_offsets, counts, d: int):
    """Move cached rows: of each request, row ``sources[i]`` to ``slots[i]`` for its first ``counts[b]``
    rows i from ``q_offsets[b]`` on, in all of ``caches`` (one launch).

    ``caches``: a cache, a list of them (256 at most, of one shape, each from ``kv4_cache``; checking them takes
    the host 0.8 us each), or one tensor [layers, ...] of the same bytes, which the caller allocates; that and its
    slices do not remember a head dim, so ``d`` has to be the one that they are used with everywhere.  ``sources`` and ``slots``
    int32 [T], ``q_offsets`` int32 [B + 1], ``counts`` int32 [B].  Rows with a source or a slot outside the cache are
    skipped.  No source may be the slot of an earlier row of its request
    or of any row of another one (``tree_accept`` gives none such)."""
    if isinstance(caches, torch.Tensor):
        index, layers = caches.get_device(), caches.dim() == 5
        pages, heads, page = _cache_shape(caches, d, 5 if layers else 4)
        n = caches.shape[0] if layers else 1
        if index < 0 or not 1 <= n <= 256:
            raise ValueError("caches must be on a CUDA device, 1 to 256 layers")
        base, size = caches.data_ptr(), caches.numel() // n
        addresses = range(base, base + n * size, size) if size else (base,) * n
    else:
        if not 1 <= len(caches) <= 256:
            raise ValueError("there must be 1 to 256 caches")
        one = caches[0]
        index, shape = one.get_device(), one.shape
        pages, heads, page = _cache_shape(one, d)
        for t in caches:
            if t.shape != shape or t.get_device() != index or index < 0:
                raise ValueError("caches must have one shape and be on one CUDA device")
            _cache_shape(t, d)
        addresses = [t.data_ptr() for t in caches]
        n = len(addresses)
        if len(set(addresses)) != n:
            raise ValueError("a cache is given twice")
    B = counts.shape[0] if counts.dim() == 1 else -1
    T = sources.shape[0] if sources.dim() == 1 else -1
    if B < 0 or T < 0:
        raise ValueError("sources and counts must be vectors")
    _ints(sources, (T,), index, "sources")
    _ints(slots, (T,), index, "slots")
    _ints(q_offsets, (B + 1,), index, "q_offsets")
    _ints(counts, (B,), index, "counts")
    if T == 0 or B == 0:
        return
    addresses = array.array("Q", addresses)  # (64 of them 1.8 us, as a ctypes array 6.5)
    _run("fa_kv4_move", index, addresses.buffer_info()[0], n, pages, page, heads, d, sources.data_ptr(),
         slots.data_ptr(), q_offsets.data_ptr(), counts.data_ptr(), T, B)


@functools.lru_cache(maxsize=1024)
def kv4_tree_workspace_bytes(Hq: int, Hkv: int, d: int, max_q: int, page_size: int, width: int) -> int:
    """Bytes of scratch ``kv4_tree_fwd`` needs for tables of ``width`` pages, whatever the lengths are (0:
    none, when no key head's work is ever split)."""
    if max(Hq, Hkv, d, page_size, width) > _most:
        return 0  # as for other invalid arguments
    return int(_fn("fa_kv4_tree_fwd_workspace_bytes")(Hq, Hkv, d, min(max_q, _most), page_size, width))


def kv4_tree_fwd(q, cache, table, lens, q_offsets, seen, max_q: int | None = None, scale: float | None = None,
                 k_descale: float = 1.0, v_descale: float = 1.0, out=None, lse=None, workspace=None,
                 status=None):
    """Attention of trees of drafted tokens (q bf16 [T, Hq, d]) over the 4-bit cache that holds them already;
    returns (o bf16 [T, Hq, d], lse fp32 [T, Hq]).

    Request b's nodes are rows q_offsets[b] .. q_offsets[b + 1) and the last tokens of its ``lens[b]`` cached
    ones, in their order.  A node sees every cached token before its tree, and of the tree's nodes those whose bit is
    set in its row of ``seen`` (int32 [T, words], words up to 8, bit i % 32 of word i / 32: node i), as
    ``tree_plan`` makes it; any other mask of bits will do.  ``max_q``: about the most nodes of a request
    (default T / B, rounded up); it only picks how many rows share a pass over the cache.  The rest as in
    ``kv4_fwd``; ``workspace``: kv4_tree_workspace_bytes(...) bytes."""
    index = q.get_device()
    if q.dtype is not _bf16 or q.dim() != 3 or index < 0:
        raise ValueError("q must be a bf16 CUDA tensor [T, Hq, d]")
    q0, q1, q2 = q.stride()
    T, Hq, d = q.shape
    pages, Hkv, page = _cache_shape(cache, d)
    if q2 != 1 or cache.get_device() != index or Hkv < 1 or Hq % Hkv:
        raise ValueError("q's last dimension must be contiguous, its heads a multiple of the cache's, "
                         "both on one device")
    if table.dim() != 2:
        raise ValueError("table must be [B, width]")
    B, width = table.shape
    _ints(table, (B, width), index, "table")
    _ints(lens, (B,), index, "lens")
    _ints(q_offsets, (B + 1,), index, "q_offsets")
    words = _seen(seen, T, index)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=_bf16, device=q.device)
    elif (out.shape != q.shape or out.dtype is not _bf16 or out.get_device() != index
          or not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 tensor shaped like q")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=_f32, device=q.device)
    elif (lse.shape != (T, Hq) or lse.dtype is not _f32 or lse.get_device() != index
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [T, Hq] tensor")
    if status is not None and (status.dtype is not _i32 or status.get_device() != index
                               or status.numel() < 1):
        raise ValueError("status must be an int32 tensor of one element on q's device")
    if T == 0:
        return out, lse
    if max_q is None:
        max_q = max(1, -(-T // max(B, 1)))
    elif max_q > _most:
        max_q = _most
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    scratch = None
    if workspace is None:
        size = kv4_tree_workspace_bytes(Hq, Hkv, d, max_q, page, width)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            scratch = workspace.data_ptr()
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        size, scratch = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _run("fa_kv4_tree_fwd", index, q.data_ptr(), q0, q1, cache.data_ptr(), pages, page, table.data_ptr(), width,
         lens.data_ptr(), q_offsets.data_ptr(), seen.data_ptr(), words, out.data_ptr(), lse.data_ptr(), T, B, Hq,
         Hkv, d, max_q, scale, k_descale, v_descale, scratch, size,
         status.data_ptr() if status is not None else None)
    return out, lse
