"""Host-side refusals of rotary positions with several axes and of the tree operators: every bad call returns a
status and launches nothing (CPU only; the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import exact_attention_13_gb300 as ea
from exact_attention_13_gb300 import _kv_abi

P = 0x10000
S3 = ctypes.c_longlong * 3
BAD, UNS, MIS = ea.FA_ERR_INVALID_ARG, ea.FA_ERR_UNSUPPORTED, ea.FA_ERR_MISALIGNED


def caches(*addresses):
    return (ctypes.c_void_p * len(addresses))(*addresses)


NAMES = {
    "fa_rope_axes": "q qs qo qos Hq k ks ko kos Hk B N d pos A posa posb axes turns r flags m stream",
    "fa_tree_plan": "parents off lens B T words pos seen stream",
    "fa_tree_accept": "parents seen words tokens choices lens new off slots table width queue size state B page T "
                      "lens_out counts path next sources state_out stream",
    "fa_kv4_move": "caches n pages page H d sources slots off counts T B stream",
    "fa_kv4_tree_fwd": "q qr qh cache pages page table width lens off seen words o lse T B Hq Hkv d max_q scale "
                       "kd vd ws ws_bytes status stream",
}
GOOD = {
    "fa_rope_axes": [P, S3(0, 128, 512), P, S3(0, 128, 512), 4, P, S3(0, 128, 128), P, S3(0, 128, 128), 1,
                     1, 8, 128, P, 3, 8, 0, P, P, 128, 0, 1.0, None],
    "fa_tree_plan": [P, P, P, 2, 8, 1, P + 64, P + 128, None],
    "fa_tree_accept": [P, P, 1, P, P, P, P, P, P, P, 4, P, 16, P, 2, 16, 8, P + 64, P + 64, P + 64, P + 64, P + 64,
                       P + 64, None],
    "fa_kv4_move": [caches(P, P + 1024), 2, 4, 16, 1, 128, P, P, P, P, 8, 2, None],
    "fa_kv4_tree_fwd": [P, 512, 128, P, 4, 16, P, 100, P, P, P, 1, P + 64, P, 8, 2, 4, 1, 128, 4, 0.1, 1.0, 1.0, P,
                        1 << 30, None, None],
}
CASES = [
    ("fa_rope_axes", dict(q=0), BAD), ("fa_rope_axes", dict(ko=0), BAD), ("fa_rope_axes", dict(pos=0), BAD),
    ("fa_rope_axes", dict(turns=0), BAD), ("fa_rope_axes", dict(axes=0), BAD), ("fa_rope_axes", dict(A=0), BAD),
    ("fa_rope_axes", dict(A=5), UNS), ("fa_rope_axes", dict(posa=-1), BAD), ("fa_rope_axes", dict(posb=-1), BAD),
    ("fa_rope_axes", dict(Hq=0), BAD), ("fa_rope_axes", dict(N=0), BAD), ("fa_rope_axes", dict(flags=4), BAD),
    ("fa_rope_axes", dict(m=float("nan")), BAD), ("fa_rope_axes", dict(d=96), UNS),
    ("fa_rope_axes", dict(r=24), UNS), ("fa_rope_axes", dict(axes=P + 4), MIS),
    ("fa_rope_axes", dict(qos=S3(0, 132, 512)), MIS), ("fa_rope_axes", dict(turns=P + 4), MIS),
    ("fa_tree_plan", dict(parents=0), BAD), ("fa_tree_plan", dict(off=0), BAD), ("fa_tree_plan", dict(seen=0), BAD),
    ("fa_tree_plan", dict(B=0), BAD), ("fa_tree_plan", dict(T=0), BAD), ("fa_tree_plan", dict(words=0), BAD),
    ("fa_tree_plan", dict(words=9), UNS), ("fa_tree_plan", dict(B=16385), UNS),
    ("fa_tree_plan", dict(T=1 << 29, words=8), UNS), ("fa_tree_plan", dict(seen=P + 2), MIS),
    ("fa_tree_accept", dict(parents=0), BAD), ("fa_tree_accept", dict(slots=0), BAD),
    ("fa_tree_accept", dict(path=0), BAD), ("fa_tree_accept", dict(queue=0), BAD),
    ("fa_tree_accept", dict(T=-1), BAD), ("fa_tree_accept", dict(B=0), BAD), ("fa_tree_accept", dict(size=0), BAD),
    ("fa_tree_accept", dict(words=0), BAD), ("fa_tree_accept", dict(lens_out=P), BAD),
    ("fa_tree_accept", dict(state_out=P), BAD), ("fa_tree_accept", dict(words=9), UNS),
    ("fa_tree_accept", dict(page=24), UNS), ("fa_tree_accept", dict(B=16385), UNS),
    ("fa_tree_accept", dict(width=1 << 27), UNS), ("fa_tree_accept", dict(B=16384, width=1 << 17), UNS),
    ("fa_tree_accept", dict(T=1 << 29, words=8), UNS), ("fa_tree_accept", dict(counts=P + 2), MIS),
    ("fa_kv4_move", dict(caches=None), BAD), ("fa_kv4_move", dict(sources=0), BAD),
    ("fa_kv4_move", dict(counts=0), BAD), ("fa_kv4_move", dict(n=0), BAD), ("fa_kv4_move", dict(T=0), BAD),
    ("fa_kv4_move", dict(B=0), BAD), ("fa_kv4_move", dict(caches=caches(P, 0)), BAD),
    ("fa_kv4_move", dict(pages=0), BAD), ("fa_kv4_move", dict(n=257, caches=caches(*[P] * 257)), UNS),
    ("fa_kv4_move", dict(d=96), UNS), ("fa_kv4_move", dict(page=8), UNS), ("fa_kv4_move", dict(pages=1 << 28), UNS),
    ("fa_kv4_move", dict(B=1 << 27, H=2), UNS), ("fa_kv4_move", dict(caches=caches(P, P + 8)), MIS),
    ("fa_kv4_move", dict(slots=P + 1), MIS),
    ("fa_kv4_tree_fwd", dict(q=0), BAD), ("fa_kv4_tree_fwd", dict(lens=0), BAD),
    ("fa_kv4_tree_fwd", dict(off=0), BAD), ("fa_kv4_tree_fwd", dict(seen=0), BAD),
    ("fa_kv4_tree_fwd", dict(words=0), BAD), ("fa_kv4_tree_fwd", dict(ws=0), BAD),
    ("fa_kv4_tree_fwd", dict(ws_bytes=1024), BAD), ("fa_kv4_tree_fwd", dict(T=0), BAD),
    ("fa_kv4_tree_fwd", dict(Hq=3, Hkv=2), BAD), ("fa_kv4_tree_fwd", dict(max_q=0), BAD),
    ("fa_kv4_tree_fwd", dict(scale=-1.0), BAD), ("fa_kv4_tree_fwd", dict(scale=float("nan")), BAD),
    ("fa_kv4_tree_fwd", dict(scale=3e38, kd=4.0), BAD), ("fa_kv4_tree_fwd", dict(kd=0.7), BAD),
    ("fa_kv4_tree_fwd", dict(width=0), BAD), ("fa_kv4_tree_fwd", dict(o=P), BAD),
    ("fa_kv4_tree_fwd", dict(d=32), UNS), ("fa_kv4_tree_fwd", dict(page=1024), UNS),
    ("fa_kv4_tree_fwd", dict(T=1 << 29), UNS), ("fa_kv4_tree_fwd", dict(words=9), UNS),
    ("fa_kv4_tree_fwd", dict(width=(1 << 26) + 1), UNS), ("fa_kv4_tree_fwd", dict(q=P + 2), MIS),
    ("fa_kv4_tree_fwd", dict(qr=100), MIS), ("fa_kv4_tree_fwd", dict(seen=P + 2), MIS),
    ("fa_kv4_tree_fwd", dict(ws=P + 8), MIS), ("fa_kv4_tree_fwd", dict(status=P + 2), MIS),
]


def test_argument_tables_match_the_signatures():
    for name, words in NAMES.items():
        assert len(words.split()) == len(_kv_abi.SIGNATURES[name][1]) == len(GOOD[name])


@pytest.mark.parametrize("fn,change,want", CASES,
                         ids=[f"{f}-{'-'.join(c)}{i}" for i, (f, c, _) in enumerate(CASES)])
def test_refusals(fn, change, want):
    args = list(GOOD[fn])
    for k, v in change.items():
        args[NAMES[fn].split().index(k)] = v
    assert getattr(ea.lib(), fn)(*args) == want


def test_workspace_sizes():
    size = ea.kv4_tree_workspace_bytes
    assert size(32, 8, 128, 16, 64, 100) > 0
    assert size(32, 8, 128, 16, 16, 1) == 0  # 16 keys: nothing is split
    for bad in ((0, 1, 128, 1), (3, 2, 128, 1), (4, 2, 96, 1), (4, 2, 128, 0)):
        assert size(*bad, 64, 100) == 0
    assert size(4, 2, 128, 1, 24, 100) == size(4, 2, 128, 1, 64, 0) == 0
    assert size(4, 2, 128, 1, 64, 1 << 24) > 0  # 2^30 tokens
    assert size(4, 2, 128, 1, 64, (1 << 24) + 1) == 0
    assert size(4, 2, 128, 1, 2 ** 32 + 64, 100) == 0
    assert size(4, 2, 128, 2 ** 40, 64, 100) == size(4, 2, 128, 2 ** 20, 64, 100)


def test_python_checks():
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i4, turns = torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.int64)
    cache = ea.kv4_cache(2, 2, 16, 128, device="cpu")
    calls = [lambda: ea.rope_axes(q, q, i4[None], turns, torch.zeros(64, dtype=torch.uint8)),
             lambda: ea.tree_plan(i4, i4[:2], i4[:1], 4),
             lambda: ea.tree_accept(i4, i4[:, None], i4, i4, i4[:1], i4[:1], i4[:2], i4, i4[None], i4, i4[:2], 16),
             lambda: ea.kv4_tree_fwd(q, cache, i4[None], i4[:1], i4[:2], i4[:, None]),
             lambda: ea.kv4_move(cache, i4, i4, i4[:2], i4[:1], 128),
             lambda: ea.kv4_move([cache], i4, i4, i4[:2], i4[:1], 128),
             lambda: ea.kv4_move([], i4, i4, i4[:2], i4[:1], 128)]
    for call in calls:  # CPU tensors are refused before the library is reached
        with pytest.raises(ValueError):
            call()
