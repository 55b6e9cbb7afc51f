"""Operators around attention: rotary positions, page planning, and the 4-bit key/value cache with
the attention that reads it.  Like the rest of the package these functions check and marshal
arguments only; the work is done by the library's CUDA kernels on the current stream.

A serving step over a paged cache, all of it on the device:

    plan = ea.page_plan(lens, new_lens, table, queue, queue_state, page_size=64, num_tokens=T)
    q, k = ea.rope(q, k, plan.positions, turns)                 # q [T, Hq, d], k [T, Hkv, d]
    ea.kv4_append(k, v, cache, plan.slots)
    o, lse = ea.kv4_fwd(q, cache, table, plan.lens, plan.q_offsets, max_q=...)

and in training, with the gradients of the rotated tensors turned back:

    qr, kr = ea.rope(q, k, positions, turns)                    # [B, H, N, d]
    o, lse = ea.fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = ea.bwd(qr, kr, v, o, lse, dout, causal=True)
    dq, dk = ea.rope(dqr, dkr, positions, turns, inverse=True)
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from ._kv_abi import FA_ROPE_INTERLEAVED, FA_ROPE_INVERSE

_strides = ctypes.c_longlong * 3


def _lib():
    from . import lib

    return lib()


def _run(fn, device, *args):
    """Call a library entry point on `device`'s current stream; raise on a status code."""
    from . import _check

    f = getattr(_lib(), fn)
    stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        _check(f(*args, stream), fn)
    else:
        with torch.cuda.device(device):
            _check(f(*args, stream), fn)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _int32(t, shape, device, name):
    _need(t.dtype == torch.int32 and t.device == device and t.is_contiguous()
          and tuple(t.shape) == shape,
          f"{name} must be a contiguous int32 tensor {list(shape)} on {device}")


# ---------------------------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------------------------
def rope_turns(rotary_dim: int, base: float = 10000.0, scaling: str | None = None,
               factor: float = 1.0, context: int = 4096, beta_fast: float = 32.0,
               beta_slow: float = 1.0, device="cuda"):
    """The frequency table of ``rope`` and the factor on rotated values: (turns, mscale).

    Pair i turns by f_i = base^(-2i / rotary_dim) per position.  ``scaling`` stretches them by
    ``factor`` for contexts longer than the ``context`` positions of training:

    * ``"linear"``: every f_i / factor (positions are interpolated)
    * ``"base"``: base * factor^(r / (r - 2)), which slows the lowest frequency by ``factor`` and
      leaves the highest
    * ``"parts"``: per pair (YaRN): f_i where a pair turns more than ``beta_fast`` times within
      ``context``, f_i / factor where it turns less than ``beta_slow`` times, a linear ramp over the
      pairs between; mscale = 0.1 ln(factor) + 1

    ``turns`` is int64, f_i / (2 pi) in units of 2^-64 turn."""
    _need(rotary_dim >= 2 and rotary_dim % 2 == 0, "rotary_dim must be even")
    _need(math.isfinite(base) and base >= 1 and math.isfinite(factor) and factor >= 1,
          "base and factor must be finite and >= 1")
    r, mscale = rotary_dim, 1.0
    if scaling == "base" and r > 2:
        base = base * factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":
        _need(context >= 1 and base > 1 and beta_fast > beta_slow > 0,
              "parts needs context >= 1, base > 1 and beta_fast > beta_slow > 0")

        def pair_that_turns(times):
            return r * math.log(context / (times * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(pair_that_turns(beta_fast)), 0)
        hi = min(math.ceil(pair_that_turns(beta_slow)), r - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
        f = [x / factor * w + x * (1 - w) for x, w in zip(f, ramp)]
        mscale = 0.1 * math.log(factor) + 1.0
    else:
        _need(scaling in (None, "base"), f"unknown scaling {scaling!r}")
    unit = 2.0 ** 64 / (2 * math.pi)
    return torch.tensor([round(x * unit) for x in f], dtype=torch.int64, device=device), mscale


def _head_strides(x, name):
    """(B, H, N, d) and {batch, head, row} strides of [B, H, N, d] or packed [T, H, d]."""
    s = x.stride()
    if x.dim() == 4:
        shape, strides = tuple(x.shape), (s[0], s[1], s[2])
    else:
        _need(x.dim() == 3, f"{name} must be [B, H, N, d] or [T, H, d]")
        shape, strides = (1, x.shape[1], x.shape[0], x.shape[2]), (0, s[1], s[0])
    _need(x.is_cuda and x.dtype == torch.bfloat16, f"{name} must be a bf16 CUDA tensor")
    _need(s[-1] == 1, f"{name}'s last dimension must be contiguous")
    return shape, strides


def rope(q, k, positions, turns, interleaved: bool = False, inverse: bool = False,
         mscale: float = 1.0, q_out=None, k_out=None):
    """Rotary positions of q and, unless it is None, k in one launch; returns (q_out, k_out).

    q, k: bf16 [B, H, N, d] (the layout of ``fwd``) or packed tokens [T, H, d], with their own
    numbers of heads; last dimension contiguous, other strides free (multiples of 8).
    ``positions``: int32 [N] or [B, N] ([T] for packed tokens).  ``turns``: int64 [rotary_dim / 2]
    from ``rope_turns``; the first rotary_dim values of a head are rotated, pairs (i, i +
    rotary_dim / 2) or, ``interleaved``, (2i, 2i + 1); the rest is copied.  ``inverse`` turns back:
    the gradients of q and k from those of the outputs, with the same ``mscale``.  ``q_out`` and
    ``k_out`` may be q and k themselves (in place)."""
    shape, qs = _head_strides(q, "q")
    B, Hq, N, d = shape
    dev = q.device
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    _need(q_out.shape == q.shape and q_out.device == dev, "q_out must match q")
    qos = _head_strides(q_out, "q_out")[1]
    Hk, kp, ko, ks, kos = 0, None, None, None, None
    if k is not None:
        kshape, ks = _head_strides(k, "k")
        Hk = kshape[1]
        _need(k.dim() == q.dim() and kshape[0] == B and kshape[2:] == (N, d) and k.device == dev,
              "k must be like q but for its heads")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=dev)
        _need(k_out.shape == k.shape and k_out.device == dev, "k_out must match k")
        kos = _strides(*_head_strides(k_out, "k_out")[1])
        ks, kp, ko = _strides(*ks), k.data_ptr(), k_out.data_ptr()
    _int32(positions, (B, N) if positions.dim() == 2 else (N,), dev, "positions")
    _need(turns.dtype == torch.int64 and turns.dim() == 1 and turns.device == dev
          and turns.is_contiguous(), f"turns must be a contiguous int64 vector on {dev}")
    _run("fa_rope", dev, q.data_ptr(), _strides(*qs), q_out.data_ptr(), _strides(*qos), Hq, kp, ks,
         ko, kos, Hk, B, N, d, positions.data_ptr(), N if positions.dim() == 2 else 0,
         turns.data_ptr(), 2 * turns.shape[0],
         (FA_ROPE_INTERLEAVED if interleaved else 0) | (FA_ROPE_INVERSE if inverse else 0),
         mscale)
    return q_out, k_out


# ---------------------------------------------------------------------------------------------
# page planning
# ---------------------------------------------------------------------------------------------
class PagePlan(NamedTuple):
    """What ``page_plan`` wrote (int32 CUDA tensors)."""

    lens: torch.Tensor         # [B] lengths after the step
    q_offsets: torch.Tensor    # [B + 1] first new token of each request
    positions: torch.Tensor    # [num_tokens]
    slots: torch.Tensor        # [num_tokens], -1: nowhere
    queue_state: torch.Tensor  # [2] head and count of the free pages after the step


def page_plan(lens, new_lens, table, queue, queue_state, page_size: int, num_tokens: int,
              out: PagePlan | None = None) -> PagePlan:
    """Pages and slots for one step of B requests, from lengths on the device (one launch).

    ``lens`` [B]: cached tokens; ``new_lens`` [B]: tokens each request brings, or -1 for one that
    has ended; ``table`` [B, width]: page ids, extended in place; ``queue`` [capacity] and
    ``queue_state`` [2] = (head, count): ring of free pages, released pages are appended in place.
    All int32.  ``num_tokens``: size of the packed batch, padding included.  Requests that do not
    get their pages keep their length and get slots of -1 (see fa_page_plan in
    include/exact_attention.h).  ``out``: a plan of the right sizes to write into; its ``lens`` and
    ``queue_state`` must not be this call's inputs."""
    dev = lens.device
    _need(lens.is_cuda and lens.dim() == 1, "lens must be an int32 CUDA vector")
    _need(table.dim() == 2 and queue.dim() == 1, "table must be [B, width], queue a vector")
    _need(num_tokens >= 0, "num_tokens must be >= 0")
    B, width = lens.shape[0], table.shape[1]
    for t, shape, name in ((lens, (B,), "lens"), (new_lens, (B,), "new_lens"),
                           (table, (B, width), "table"), (queue, tuple(queue.shape), "queue"),
                           (queue_state, (2,), "queue_state")):
        _int32(t, shape, dev, name)
    if out is None:
        # one allocation, each part on a 16-byte boundary
        sizes = (B, B + 1, num_tokens, num_tokens, 2)
        flat = torch.empty(sum(-(-n // 4) * 4 for n in sizes), dtype=torch.int32, device=dev)
        parts, at = [], 0
        for n in sizes:
            parts.append(flat[at:at + n])
            at += -(-n // 4) * 4
        out = PagePlan(*parts)
    else:
        for t, n, name in zip(out, (B, B + 1, num_tokens, num_tokens, 2), PagePlan._fields):
            _int32(t, (n,), dev, f"out.{name}")
    _run("fa_page_plan", dev, lens.data_ptr(), new_lens.data_ptr(), table.data_ptr(), width,
         queue.data_ptr(), queue.shape[0], queue_state.data_ptr(), B, page_size, num_tokens,
         out.lens.data_ptr(), out.q_offsets.data_ptr(), out.positions.data_ptr(),
         out.slots.data_ptr(), out.queue_state.data_ptr())
    return out


# ---------------------------------------------------------------------------------------------
# the 4-bit cache
# ---------------------------------------------------------------------------------------------
def kv4_cache(num_pages: int, heads: int, page_size: int, d: int, device="cuda"):
    """An empty 4-bit cache: uint8 zeros [num_pages, heads, 2, page_size * 9 d / 16]."""
    total = int(_lib().fa_kv4_cache_bytes(num_pages, heads, page_size, d))
    _need(total > 0, f"unsupported cache (pages {num_pages}, heads {heads}, page size {page_size},"
                     f" d {d})")
    return torch.zeros((num_pages, heads, 2, total // (2 * num_pages * heads)), dtype=torch.uint8,
                       device=device)


def _cache_shape(cache, d):
    """(pages, heads, page size) of a cache of head dim d."""
    _need(cache.is_cuda and cache.dtype == torch.uint8 and cache.dim() == 4 and cache.shape[2] == 2
          and cache.is_contiguous() and cache.shape[3] * 16 % (9 * d) == 0,
          f"cache must be a contiguous uint8 CUDA tensor as kv4_cache makes it for d = {d}")
    return cache.shape[0], cache.shape[1], cache.shape[3] * 16 // (9 * d)


def kv4_append(k, v, cache, slots, k_descale: float = 1.0, v_descale: float = 1.0):
    """Quantise k and v (bf16 [T, H, d], last dimension contiguous) and write them into the cache
    at ``slots`` (int32 [T]; rows with a slot outside the cache, such as -1, are skipped).  Descales
    are powers of two: values are stored divided by them."""
    _need(k.is_cuda and k.dtype == torch.bfloat16 and k.dim() == 3 and k.shape == v.shape
          and v.dtype == k.dtype and v.device == k.device,
          "k and v must be bf16 CUDA tensors of one shape [T, H, d]")
    ks, vs = k.stride(), v.stride()
    _need(ks[2] == 1 and vs[2] == 1, "the last dimension of k and v must be contiguous")
    T, H, d = k.shape
    pages, heads, page = _cache_shape(cache, d)
    _need(heads == H and cache.device == k.device, "the cache must have k's heads and device")
    _int32(slots, (T,), k.device, "slots")
    _run("fa_kv4_append", k.device, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
         cache.data_ptr(), pages, page, slots.data_ptr(), T, H, d, k_descale, v_descale)


def kv4_read(cache, slots, d: int, k_descale: float = 1.0, v_descale: float = 1.0, k=None, v=None):
    """The cached keys and values at ``slots`` (int32 [T]) as bf16 [T, H, d] (exact); rows whose slot
    lies outside the cache are zeros.  Returns (k, v)."""
    _need(d in (64, 128), "d must be 64 or 128")
    pages, heads, page = _cache_shape(cache, d)
    dev = cache.device
    _need(slots.dim() == 1, "slots must be a vector")
    T = slots.shape[0]
    _int32(slots, (T,), dev, "slots")
    outs = []
    for name, t in (("k", k), ("v", v)):
        if t is None:
            t = torch.empty((T, heads, d), dtype=torch.bfloat16, device=dev)
        _need(tuple(t.shape) == (T, heads, d) and t.dtype == torch.bfloat16 and t.device == dev
              and t.is_contiguous(), f"{name} must be a contiguous bf16 [T, H, d] tensor")
        outs.append(t)
    _run("fa_kv4_read", dev, cache.data_ptr(), pages, page, slots.data_ptr(), outs[0].data_ptr(),
         outs[1].data_ptr(), T, heads, d, k_descale, v_descale)
    return outs[0], outs[1]


def kv4_workspace_bytes(Hq: int, Hkv: int, d: int, max_q: int = 1) -> int:
    """Bytes of scratch ``kv4_fwd`` needs (whatever the lengths are)."""
    return int(_lib().fa_kv4_fwd_workspace_bytes(Hq, Hkv, d, max_q))


def kv4_fwd(q, cache, table, lens, q_offsets=None, max_q: int | None = None, causal: bool = True,
            scale: float | None = None, k_descale: float = 1.0, v_descale: float = 1.0, out=None,
            lse=None, workspace=None):
    """Attention of packed query tokens q (bf16 [T, Hq, d]) over the 4-bit cache; returns (o bf16
    [T, Hq, d], lse fp32 [T, Hq]).

    ``table`` int32 [B, width] and ``lens`` int32 [B] (the new tokens included) say where the keys
    are; request b's queries are rows q_offsets[b] .. q_offsets[b + 1) (int32 [B + 1]), or T / B rows
    each without ``q_offsets``.  ``causal``: the queries are the last tokens of the cache.
    ``max_q``: about the most queries of a request (default T / B, rounded up); it only picks how many
    rows share a pass over the cache.  Rows of q past the last request's are left as they are.
    ``workspace``: a CUDA tensor of kv4_workspace_bytes(...) bytes, not shared by calls that may run
    at the same time; without it torch allocates one."""
    _need(q.is_cuda and q.dtype == torch.bfloat16 and q.dim() == 3,
          "q must be a bf16 CUDA tensor [T, Hq, d]")
    qs = q.stride()
    _need(qs[2] == 1, "q's last dimension must be contiguous")
    T, Hq, d = q.shape
    dev = q.device
    _need(d in (64, 128), "d must be 64 or 128")
    pages, Hkv, page = _cache_shape(cache, d)
    _need(cache.device == dev and Hq % Hkv == 0, "q's heads must be a multiple of the cache's")
    _need(table.dim() == 2, "table must be [B, width]")
    B, width = table.shape
    _int32(table, (B, width), dev, "table")
    _int32(lens, (B,), dev, "lens")
    if q_offsets is not None:
        _int32(q_offsets, (B + 1,), dev, "q_offsets")
    else:
        _need(B > 0 and T % B == 0, "without q_offsets T must be a multiple of B")
    if max_q is None:
        max_q = max(1, -(-T // max(B, 1)))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    _need(out.shape == q.shape and out.dtype == torch.bfloat16 and out.is_contiguous()
          and out.device == dev, "out must be a contiguous bf16 tensor shaped like q")
    _need(tuple(lse.shape) == (T, Hq) and lse.dtype == torch.float32 and lse.is_contiguous()
          and lse.device == dev, "lse must be a contiguous fp32 [T, Hq] tensor")
    if workspace is None:
        workspace = torch.empty(kv4_workspace_bytes(Hq, Hkv, d, max_q), dtype=torch.uint8,
                                device=dev)
    _need(workspace.device == dev and workspace.is_contiguous(),
          "workspace must be a contiguous tensor on q's device")
    _run("fa_kv4_fwd", dev, q.data_ptr(), qs[0], qs[1], cache.data_ptr(), pages, page,
         table.data_ptr(), width, lens.data_ptr(),
         q_offsets.data_ptr() if q_offsets is not None else None, out.data_ptr(), lse.data_ptr(),
         T, B, Hq, Hkv, d, max_q, scale, bool(causal), k_descale, v_descale, workspace.data_ptr(),
         workspace.numel() * workspace.element_size())
    return out, lse
