"""Operators around attention: rotary positions, page planning, and the 4-bit key/value cache with
the attention that reads it.  Like the rest of the package these functions check and marshal
arguments only; the work is done by the library's CUDA kernels on the current stream.

A serving step over a paged cache, all of it on the device:

    plan = ea.page_plan(lens, new_lens, table, queue, queue_state, page_size=64, num_tokens=T)
    q, k = ea.rope(q, k, plan.positions, turns)                 # q [T, Hq, d], k [T, Hkv, d]
    ea.kv4_append(k, v, cache, plan.slots)
    o, lse = ea.kv4_fwd(q, cache, table, plan.lens, plan.q_offsets, max_q=...)

A step without tokens (T = 0, as when all requests have just ended) passes through all of them: calls on
no rows check their tensors and launch nothing.

And in training, with the gradients of the rotated tensors turned back:

    qr, kr = ea.rope(q, k, positions, turns)                    # [B, H, N, d]
    o, lse = ea.fwd(qr, kr, v, causal=True)
    dqr, dkr, dv = ea.bwd(qr, kr, v, o, lse, dout, causal=True)
    dq, dk = ea.rope(dqr, dkr, positions, turns, inverse=True)
"""
from __future__ import annotations

import ctypes
import decimal
import functools
import math
from typing import NamedTuple

import torch

from . import _check, lib
from ._kv_abi import FA_ROPE_INTERLEAVED, FA_ROPE_INVERSE

_bf16, _i32, _f32 = torch.bfloat16, torch.int32, torch.float32
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_bound = {}
_most = 0x7fffffff  # the library's sizes are 32 bits, and ctypes drops what lies above them


def _fn(name):
    """The library's entry point (looked up once: these calls are made once per layer and token)."""
    f = _bound.get(name)
    if f is None:
        f = _bound[name] = getattr(lib(), name)
    return f


def _run(name, index, *args):
    """Call an entry point on device `index`'s current stream; raise on a status code."""
    f = _bound.get(name) or _fn(name)
    if index == _current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc:
        _check(rc, name)


@functools.lru_cache(maxsize=1024)
def _strides(batch, head, row):
    """A C array of three strides (only ever read)."""
    return (ctypes.c_longlong * 3)(batch, head, row)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(t, shape, index, name):
    if (t.dtype is not _i32 or t.get_device() != index or t.shape != shape
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on cuda:{index}")
    if shape[0] > _most or shape[-1] > _most:
        raise ValueError(f"{name} has a side of more than 2^31 - 1 entries")


# ---------------------------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------------------------
_PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510")


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

    ``turns`` is int64, f_i / (2 pi) in units of 2^-64 turn, rounded to nearest: computed with 50 digits,
    because the 53 bits of a double leave an error of up to 2^9 units."""
    _need(rotary_dim >= 2 and rotary_dim % 2 == 0, "rotary_dim must be even")
    _need(math.isfinite(base) and base >= 1 and math.isfinite(factor) and factor >= 1,
          "base and factor must be finite and >= 1")
    r, mscale = int(rotary_dim), 1.0
    exact = decimal.Context(prec=50)
    base_x, factor_x = decimal.Decimal(float(base)), decimal.Decimal(float(factor))
    with decimal.localcontext(exact):
        if scaling == "base" and r > 2:
            base_x *= factor_x ** (decimal.Decimal(r) / (r - 2))
        f = [base_x ** (decimal.Decimal(-2 * i) / r) for i in range(r // 2)]
        if scaling == "linear":
            f = [x / factor_x for x in f]
        elif scaling == "parts":
            _need(context >= 1 and base > 1 and beta_fast > beta_slow > 0,
                  "parts needs context >= 1, base > 1 and beta_fast > beta_slow > 0")

            def pair_that_turns(times):
                return r * math.log(context / (times * 2 * math.pi)) / (2 * math.log(base))

            lo = max(math.floor(pair_that_turns(beta_fast)), 0)
            hi = min(math.ceil(pair_that_turns(beta_slow)), r - 1)
            width = decimal.Decimal(hi - lo) if hi > lo else decimal.Decimal("1e-3")
            ramp = [min(max((i - lo) / width, 0), 1) for i in range(r // 2)]
            f = [x / factor_x * w + x * (1 - w) for x, w in zip(f, ramp)]
            mscale = 0.1 * math.log(factor) + 1.0
        else:
            _need(scaling in (None, "base"), f"unknown scaling {scaling!r}")
        unit = 2 ** 64 / (2 * _PI)
        turns = [int((x * unit).to_integral_value(decimal.ROUND_HALF_EVEN)) for x in f]
    return torch.tensor(turns, dtype=torch.int64, device=device), mscale


def _heads(x, index, name):
    """(B, H, N, d) and the {batch, head, row} strides of [B, H, N, d] or packed [T, H, d]."""
    if x.dtype is not _bf16 or x.get_device() != index or index < 0:
        raise ValueError(f"{name} must be a bf16 CUDA tensor, all on one device")
    shape, s = x.shape, x.stride()
    if len(shape) == 4:
        strides = _strides(s[0], s[1], s[2])
    elif len(shape) == 3:
        shape, strides = (1, shape[1], shape[0], shape[2]), _strides(0, s[1], s[0])
    else:
        raise ValueError(f"{name} must be [B, H, N, d] or [T, H, d]")
    if s[-1] != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return shape, strides


def _out_like(x, out, index, name):
    """`out`, or a new contiguous tensor like x, and its strides."""
    if out is None:
        out = torch.empty(x.shape, dtype=_bf16, device=x.device)
        s = out.stride()
        return out, _strides(*s[:3]) if len(s) == 4 else _strides(0, s[1], s[0])
    if out.shape != x.shape:
        raise ValueError(f"{name} must have its input's shape")
    return out, _heads(out, index, name)[1]


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
    index = q.get_device()
    (B, Hq, N, d), qs = _heads(q, index, "q")
    q_out, qos = _out_like(q, q_out, index, "q_out")
    if k is None:
        k_out, Hk, kp, ko, ks, kos = None, 0, None, None, None, None
    else:
        (Bk, Hk, Nk, dk), ks = _heads(k, index, "k")
        if Bk != B or Nk != N or dk != d or k.dim() != q.dim():
            raise ValueError("k must be like q but for its heads")
        k_out, kos = _out_like(k, k_out, index, "k_out")
        kp, ko = k.data_ptr(), k_out.data_ptr()
    per_batch = positions.dim() == 2
    _ints(positions, (B, N) if per_batch else (N,), index, "positions")
    if (turns.dtype is not torch.int64 or turns.dim() != 1 or turns.get_device() != index
            or not turns.is_contiguous()):
        raise ValueError(f"turns must be a contiguous int64 vector on cuda:{index}")
    if B * N == 0:
        return q_out, k_out
    _run("fa_rope", index, q.data_ptr(), qs, q_out.data_ptr(), qos, Hq, kp, ks, ko, kos, Hk, B, N,
         d, positions.data_ptr(), N if per_batch else 0, turns.data_ptr(), 2 * turns.shape[0],
         (FA_ROPE_INTERLEAVED if interleaved else 0) | (FA_ROPE_INVERSE if inverse else 0),
         mscale)
    return q_out, k_out


def rope_axis_pairs(sections, cycled: bool = False, device="cuda"):
    """The axis of each pair for ``rope_axes``: uint8 [sum(sections)].

    ``sections``: how many pairs each axis has, up to four axes, as (16, 24, 24) for time, height and width
    at a rotary dim of 128.  The axes take their pairs one section behind the other, or, ``cycled``, in turn
    until their sections are used up (0, 1, 2, 0, 1, 2, ...)."""
    left = [int(n) for n in sections]
    _need(1 <= len(left) <= 4 and all(n >= 0 for n in left) and 0 < sum(left) <= 64,
          "sections must be the pairs of one to four axes, 64 in all at most")
    if cycled:
        pairs = [a for i in range(max(left)) for a, n in enumerate(left) if i < n]
    else:
        pairs = [a for a, n in enumerate(left) for _ in range(n)]
    return torch.tensor(pairs, dtype=torch.uint8, device=device)


def rope_axes(q, k, positions, turns, axes, interleaved: bool = False, inverse: bool = False,
              mscale: float = 1.0, q_out=None, k_out=None):
    """Rotary positions with several axes (the time, height and width of image and video tokens): as
    ``rope``, but pair i turns by position ``axes[i]`` of its token.

    ``positions``: int32 [A, N] or [A, B, N] ([A, T] for packed tokens), A from 1 to 4; text tokens have the
    same position on all axes.  ``axes``: uint8 [rotary_dim / 2], as ``rope_axis_pairs`` makes it (an axis
    that there is not counts as the first).  ``turns``: from ``rope_turns``, or any table that gives each pair its own
    frequency.  ``inverse``: the gradients of q and k from those of the outputs."""
    index = q.get_device()
    (B, Hq, N, d), qs = _heads(q, index, "q")
    q_out, qos = _out_like(q, q_out, index, "q_out")
    if k is None:
        k_out, Hk, kp, ko, ks, kos = None, 0, None, None, None, None
    else:
        (Bk, Hk, Nk, dk), ks = _heads(k, index, "k")
        if Bk != B or Nk != N or dk != d or k.dim() != q.dim():
            raise ValueError("k must be like q but for its heads")
        k_out, kos = _out_like(k, k_out, index, "k_out")
        kp, ko = k.data_ptr(), k_out.data_ptr()
    shape = positions.shape
    per_batch = len(shape) == 3
    if not 2 <= len(shape) <= 3 or not 1 <= shape[0] <= 4:
        raise ValueError("positions must be [axes, N] or [axes, B, N] with one to four axes")
    _ints(positions, (shape[0], B, N) if per_batch else (shape[0], N), index, "positions")
    if (turns.dtype is not torch.int64 or turns.dim() != 1 or turns.get_device() != index
            or not turns.is_contiguous()):
        raise ValueError(f"turns must be a contiguous int64 vector on cuda:{index}")
    if (axes.dtype is not torch.uint8 or axes.shape != turns.shape or axes.get_device() != index
            or not axes.is_contiguous()):
        raise ValueError(f"axes must be a contiguous uint8 vector as long as turns on cuda:{index}")
    if B * N == 0:
        return q_out, k_out
    _run("fa_rope_axes", index, q.data_ptr(), qs, q_out.data_ptr(), qos, Hq, kp, ks, ko, kos, Hk, B, N, d,
         positions.data_ptr(), shape[0], B * N if per_batch else N, N if per_batch else 0, axes.data_ptr(),
         turns.data_ptr(), 2 * turns.shape[0],
         (FA_ROPE_INTERLEAVED if interleaved else 0) | (FA_ROPE_INVERSE if inverse else 0), mscale)
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
    All int32, B from 1 to 16384.  ``num_tokens``: size of the packed batch, padding included.  Requests that
    do not get their pages keep their length and get slots of -1; what attention gives for their tokens means
    nothing (see fa_page_plan in include/exact_attention.h).  ``out``: a plan of the right sizes to write into; its ``lens`` and
    ``queue_state`` must not be this call's inputs."""
    index = lens.get_device()
    if (index < 0 or lens.dim() != 1 or table.dim() != 2 or queue.dim() != 1
            or not 0 <= num_tokens <= _most or not 0 < page_size <= _most):
        raise ValueError("lens and queue must be int32 CUDA vectors, table [B, width], num_tokens in "
                         "[0, 2^31), page_size in (0, 2^31)")
    B, width, cap = lens.shape[0], table.shape[1], queue.shape[0]
    _ints(lens, (B,), index, "lens")
    _ints(new_lens, (B,), index, "new_lens")
    _ints(table, (B, width), index, "table")
    _ints(queue, (cap,), index, "queue")
    _ints(queue_state, (2,), index, "queue_state")
    sizes = (B, B + 1, num_tokens, num_tokens, 2)
    if out is None:
        # one allocation for the five parts (integers: nothing tracks these views; 8.5 us on the host,
        # of the 12.3 of tracked ones and the 12.5 of five allocations)
        flat = torch.empty(2 * (B + num_tokens) + 3, dtype=_i32, device=lens.device)
        out = PagePlan._make(torch.unsafe_split_with_sizes(flat, sizes))
    else:
        for t, n, name in zip(out, sizes, PagePlan._fields):
            _ints(t, (n,), index, f"out.{name}")
    _run("fa_page_plan", index, lens.data_ptr(), new_lens.data_ptr(), table.data_ptr(), width,
         queue.data_ptr(), cap, queue_state.data_ptr(), B, page_size, num_tokens,
         out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
         out[4].data_ptr())
    return out


# ---------------------------------------------------------------------------------------------
# the 4-bit cache
# ---------------------------------------------------------------------------------------------
def kv4_cache(num_pages: int, heads: int, page_size: int, d: int, device="cuda"):
    """An empty 4-bit cache: uint8 zeros [num_pages, heads, 2, page_size * 9 d / 16].

    The bytes alone do not tell pages of 128 tokens with d = 64 from pages of 64 tokens with d = 128 (or 64
    from 32, 32 from 16).  The tensor returned here remembers its d, and calls with the other one are
    refused; on its views and copies the caller has to keep to d."""
    total = 0
    if all(0 < n <= _most for n in (num_pages, heads, page_size, d)):
        total = int(_fn("fa_kv4_cache_bytes")(num_pages, heads, page_size, d))
    _need(total > 0, f"unsupported cache (pages {num_pages}, heads {heads}, page size {page_size},"
                     f" d {d})")
    cache = torch.zeros((num_pages, heads, 2, total // (2 * num_pages * heads)), dtype=torch.uint8,
                        device=device)
    cache._kv4_d = d
    return cache


def _cache_shape(cache, d, dims=4):
    """(pages, heads, page size) of a cache of head dim d (5 dims: of several in one tensor)."""
    if cache.dim() != dims or d < 16:
        raise ValueError("cache must be as kv4_cache makes it")
    pages, heads, two, block = cache.shape if dims == 4 else cache.shape[1:]
    page, rest = divmod(block * 16, 9 * d)
    if rest or two != 2 or cache.dtype is not torch.uint8 or not cache.is_contiguous():
        raise ValueError(f"cache must be a contiguous uint8 tensor as kv4_cache makes it for d = {d}")
    if getattr(cache, "_kv4_d", d) != d:
        raise ValueError(f"the cache was made for d = {cache._kv4_d}, not {d}")
    return pages, heads, page


def kv4_append(k, v, cache, slots, k_descale: float = 1.0, v_descale: float = 1.0):
    """Quantise k and v (bf16 [T, H, d], last dimension contiguous) and write them into the cache
    at ``slots`` (int32 [T]; rows with a slot outside the cache, such as -1, are skipped).  Descales
    are powers of two: values are stored divided by them.  A group of 16 values keeps its precision where its
    largest, so divided, lies between 0.1 and 2688 (6 times e4m3's normal range); below the scale gets coarse,
    below 0.006 the group is stored as zeros, above 2688 it saturates."""
    index = k.get_device()
    if (k.dtype is not _bf16 or v.dtype is not _bf16 or k.dim() != 3 or k.shape != v.shape
            or index < 0 or v.get_device() != index):
        raise ValueError("k and v must be bf16 CUDA tensors of one shape [T, H, d]")
    (k0, k1, k2), (v0, v1, v2) = k.stride(), v.stride()
    if k2 != 1 or v2 != 1:
        raise ValueError("the last dimension of k and v must be contiguous")
    T, H, d = k.shape
    pages, heads, page = _cache_shape(cache, d)
    if heads != H or cache.get_device() != index:
        raise ValueError("the cache must have k's heads and device")
    _ints(slots, (T,), index, "slots")
    if T == 0:
        return
    _run("fa_kv4_append", index, k.data_ptr(), k0, k1, v.data_ptr(), v0, v1, cache.data_ptr(),
         pages, page, slots.data_ptr(), T, H, d, k_descale, v_descale)


def kv4_read(cache, slots, d: int, k_descale: float = 1.0, v_descale: float = 1.0, k=None, v=None):
    """The cached keys and values at ``slots`` (int32 [T]) as bf16 [T, H, d] (exact); rows whose slot
    lies outside the cache are zeros.  Returns (k, v)."""
    index = cache.get_device()
    pages, heads, page = _cache_shape(cache, d)
    if index < 0 or slots.dim() != 1:
        raise ValueError("the cache must be on a CUDA device, slots a vector")
    T = slots.shape[0]
    _ints(slots, (T,), index, "slots")
    shape = (T, heads, d)
    if k is None:
        k = torch.empty(shape, dtype=_bf16, device=cache.device)
    if v is None:
        v = torch.empty(shape, dtype=_bf16, device=cache.device)
    for t in (k, v):
        if (t.shape != shape or t.dtype is not _bf16 or t.get_device() != index
                or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous bf16 [T, H, d] tensors")
    if T == 0:
        return k, v
    _run("fa_kv4_read", index, cache.data_ptr(), pages, page, slots.data_ptr(), k.data_ptr(),
         v.data_ptr(), T, heads, d, k_descale, v_descale)
    return k, v


@functools.lru_cache(maxsize=1024)
def kv4_workspace_bytes(Hq: int, Hkv: int, d: int, max_q: int, page_size: int, width: int) -> int:
    """Bytes of scratch ``kv4_fwd`` needs for tables of ``width`` pages, whatever the lengths are
    (0: none, when no key head's work is ever split)."""
    if max(Hq, Hkv, d, page_size, width) > _most:
        return 0  # as for other invalid arguments
    return int(_fn("fa_kv4_fwd_workspace_bytes")(Hq, Hkv, d, min(max_q, _most), page_size, width))


def kv4_fwd(q, cache, table, lens, q_offsets=None, max_q: int | None = None, causal: bool = True,
            scale: float | None = None, k_descale: float = 1.0, v_descale: float = 1.0, out=None,
            lse=None, workspace=None, status=None):
    """Attention of packed query tokens q (bf16 [T, Hq, d]) over the 4-bit cache; returns (o bf16
    [T, Hq, d], lse fp32 [T, Hq]).

    ``table`` int32 [B, width] and ``lens`` int32 [B] (the new tokens included) say where the keys
    are; request b's queries are rows q_offsets[b] .. q_offsets[b + 1) (int32 [B + 1]), or T / B rows
    each without ``q_offsets``.  ``causal``: the queries are the last tokens of the cache.
    ``max_q``: about the most queries of a request (default T / B, rounded up); it only picks the
    kernel (how many rows share a pass over the cache), one for all requests of the call.  Drafts of several
    requests with 17 to 128 query rows a key head take less time at d = 128 as chains through ``kv4_tree_fwd`` (64
    requests of 4096 keys: 123 us instead of 163 for 32 rows, 141 instead of 229 for 64).  Rows of ``out`` and
    ``lse`` past the last request's are left as they are (not initialised in tensors made here).  Rows of
    tokens without a slot, such as those of a request that ``page_plan`` refused, mean nothing: their keys are
    not in the cache, and they see what it held before.
    ``workspace``: a CUDA tensor of kv4_workspace_bytes(...) bytes or more, not shared by calls that may run
    at the same time; without it torch allocates one.  ``status``: as in ``fwd``."""
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
    offsets = None
    if q_offsets is not None:
        _ints(q_offsets, (B + 1,), index, "q_offsets")
        offsets = q_offsets.data_ptr()
    elif B < 1 or T % B:
        raise ValueError("without q_offsets T must be a multiple of B")
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
        size = kv4_workspace_bytes(Hq, Hkv, d, max_q, page, width)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            scratch = workspace.data_ptr()
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        size, scratch = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _run("fa_kv4_fwd", index, q.data_ptr(), q0, q1, cache.data_ptr(), pages, page,
         table.data_ptr(), width, lens.data_ptr(), offsets, out.data_ptr(), lse.data_ptr(), T, B,
         Hq, Hkv, d, max_q, scale, 1 if causal else 0, k_descale, v_descale, scratch, size,
         status.data_ptr() if status is not None else None)
    return out, lse
