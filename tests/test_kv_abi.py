"""Host-side refusals of the operators around attention: every bad call returns a status and
launches nothing (CPU only; the addresses are never dereferenced)."""
import ctypes

import pytest
import torch

import exact_attention_13_gb300 as ea
from exact_attention_13_gb300 import _kv_abi

P = 0x10000
S3 = ctypes.c_longlong * 3
BAD, UNS, MIS = ea.FA_ERR_INVALID_ARG, ea.FA_ERR_UNSUPPORTED, ea.FA_ERR_MISALIGNED

NAMES = {
    "fa_rope": "q qs qo qos Hq k ks ko kos Hk B N d pos posb turns r flags m stream",
    "fa_page_plan": "lens new table width queue size state B page T lens_out off pos slots state_out "
                    "stream",
    "fa_kv4_append": "k kr kh v vr vh cache pages page slots T H d kd vd stream",
    "fa_kv4_read": "cache pages page slots k v T H d kd vd stream",
    "fa_kv4_fwd": "q qr qh cache pages page table width lens off o lse T B Hq Hkv d max_q scale "
                  "causal kd vd ws ws_bytes status stream",
}
GOOD = {
    "fa_rope": [P, S3(0, 128, 512), P, S3(0, 128, 512), 4, P, S3(0, 128, 128), P, S3(0, 128, 128), 1,
                1, 8, 128, P, 0, P, 128, 0, 1.0, None],
    "fa_page_plan": [P, P, P, 4, P, 16, P, 2, 16, 8, P + 64, P, P, P, P + 64, None],
    "fa_kv4_append": [P, 128, 128, P, 128, 128, P, 4, 16, P, 8, 1, 128, 1.0, 1.0, None],
    "fa_kv4_read": [P, 4, 16, P, P, P + 64, 8, 1, 128, 1.0, 1.0, None],
    "fa_kv4_fwd": [P, 512, 128, P, 4, 16, P, 100, P, P, P + 64, P, 8, 2, 4, 1, 128, 4, 0.1, 1, 1.0, 1.0, P,
                   1 << 30, None, None],
}
CASES = [
    ("fa_rope", dict(q=0), BAD), ("fa_rope", dict(ko=0), BAD), ("fa_rope", dict(pos=0), BAD),
    ("fa_rope", dict(turns=0), BAD), ("fa_rope", dict(qs=None), BAD), ("fa_rope", dict(Hq=0), BAD),
    ("fa_rope", dict(Hk=-1), BAD), ("fa_rope", dict(N=0), BAD), ("fa_rope", dict(flags=4), BAD),
    ("fa_rope", dict(m=float("nan")), BAD), ("fa_rope", dict(posb=-1), BAD),
    ("fa_rope", dict(qs=S3(0, -128, 512)), BAD), ("fa_rope", dict(d=96), UNS),
    ("fa_rope", dict(r=24), UNS), ("fa_rope", dict(r=144), UNS), ("fa_rope", dict(r=0), UNS),
    ("fa_rope", dict(Hq=65535), UNS), ("fa_rope", dict(q=P + 8), MIS),
    ("fa_rope", dict(qos=S3(0, 132, 512)), MIS), ("fa_rope", dict(turns=P + 4), MIS),
    ("fa_page_plan", dict(lens=0), BAD), ("fa_page_plan", dict(queue=0), BAD),
    ("fa_page_plan", dict(slots=0), BAD), ("fa_page_plan", dict(B=0), BAD),
    ("fa_page_plan", dict(T=-1), BAD), ("fa_page_plan", dict(size=0), BAD),
    ("fa_page_plan", dict(lens_out=P), BAD), ("fa_page_plan", dict(state_out=P), BAD),
    ("fa_page_plan", dict(B=16385), UNS), ("fa_page_plan", dict(page=24), UNS),
    ("fa_page_plan", dict(page=256), UNS), ("fa_page_plan", dict(width=1 << 27), UNS),
    ("fa_page_plan", dict(B=16384, width=1 << 17), UNS), ("fa_page_plan", dict(table=P + 2), MIS),
    ("fa_kv4_append", dict(k=0), BAD), ("fa_kv4_append", dict(slots=0), BAD),
    ("fa_kv4_append", dict(cache=0), BAD), ("fa_kv4_append", dict(T=0), BAD),
    ("fa_kv4_append", dict(vr=-8), BAD), ("fa_kv4_append", dict(kd=3.0), BAD),
    ("fa_kv4_append", dict(vd=0.0), BAD), ("fa_kv4_append", dict(vd=float("inf")), BAD),
    ("fa_kv4_append", dict(kd=-1.0), BAD), ("fa_kv4_append", dict(d=256), UNS),
    ("fa_kv4_append", dict(page=8), UNS), ("fa_kv4_append", dict(pages=1 << 28), UNS),
    ("fa_kv4_append", dict(cache=P + 8), MIS), ("fa_kv4_append", dict(kh=129), MIS),
    ("fa_kv4_read", dict(k=0), BAD), ("fa_kv4_read", dict(T=0), BAD),
    ("fa_kv4_read", dict(kd=0.3), BAD), ("fa_kv4_read", dict(page=48), UNS),
    ("fa_kv4_read", dict(v=P + 4), MIS), ("fa_kv4_read", dict(v=P + 32, k=P + 32), BAD),
    ("fa_kv4_fwd", dict(q=0), BAD), ("fa_kv4_fwd", dict(lens=0), BAD),
    ("fa_kv4_fwd", dict(ws=0), BAD), ("fa_kv4_fwd", dict(ws_bytes=1024), BAD),
    ("fa_kv4_fwd", dict(T=0), BAD), ("fa_kv4_fwd", dict(Hq=3, Hkv=2), BAD),
    ("fa_kv4_fwd", dict(off=None, T=7), BAD), ("fa_kv4_fwd", dict(max_q=0), BAD),
    ("fa_kv4_fwd", dict(scale=-1.0), BAD), ("fa_kv4_fwd", dict(scale=float("nan")), BAD),
    ("fa_kv4_fwd", dict(scale=3e38, kd=4.0), BAD), ("fa_kv4_fwd", dict(kd=0.7), BAD),
    ("fa_kv4_fwd", dict(width=0), BAD), ("fa_kv4_fwd", dict(d=32), UNS),
    ("fa_kv4_fwd", dict(page=1024), UNS), ("fa_kv4_fwd", dict(T=1 << 29), UNS),
    ("fa_kv4_fwd", dict(q=P + 2), MIS), ("fa_kv4_fwd", dict(qr=100), MIS),
    ("fa_kv4_fwd", dict(lse=P + 2), MIS), ("fa_kv4_fwd", dict(ws=P + 8), MIS),
    ("fa_kv4_fwd", dict(o=P), BAD), ("fa_kv4_fwd", dict(width=(1 << 26) + 1), UNS),
    ("fa_kv4_fwd", dict(status=P + 2), MIS), ("fa_kv4_fwd", dict(max_q=64, ws_bytes=1 << 20), BAD),
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


def test_sizes():
    lib = ea.lib()
    assert lib.fa_kv4_cache_bytes(3, 2, 16, 128) == 3 * 2 * 2 * 16 * (64 + 8)
    assert lib.fa_kv4_cache_bytes(1 << 20, 64, 128, 128) == (1 << 20) * 64 * 2 * 128 * 72
    for bad in ((0, 1, 16, 128), (1, 0, 16, 128), (1, 1, 20, 128), (1, 1, 16, 96)):
        assert lib.fa_kv4_cache_bytes(*bad) == 0
    assert ea.kv4_workspace_bytes(32, 8, 128, 1, 64, 9) > 0
    assert ea.kv4_workspace_bytes(32, 8, 128, 1, 64, 8) == 0  # 512 keys: nothing is split
    for bad in ((0, 1, 128, 1), (3, 2, 128, 1), (4, 2, 96, 1), (4, 2, 128, 0)):
        assert ea.kv4_workspace_bytes(*bad, 64, 100) == 0
    assert ea.kv4_workspace_bytes(4, 2, 128, 1, 24, 100) == 0
    assert ea.kv4_workspace_bytes(4, 2, 128, 1, 64, 0) == 0
    assert ea.kv4_workspace_bytes(4, 2, 128, 1, 64, 1 << 24) > 0  # 2^30 tokens
    assert ea.kv4_workspace_bytes(4, 2, 128, 1, 64, (1 << 24) + 1) == 0


def test_python_checks():
    q, k = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i4, turns = torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.int64)
    cache = ea.kv4_cache(2, 2, 16, 128, device="cpu")
    assert cache.shape == (2, 2, 2, 16 * 72)
    calls = [lambda: ea.rope(q, k, i4, turns),
             lambda: ea.page_plan(i4, i4, i4[None], i4, i4[:2], 16, 4),
             lambda: ea.kv4_append(k, k, cache, i4),
             lambda: ea.kv4_read(cache, i4, 128),
             lambda: ea.kv4_fwd(q, cache, i4[None], i4[:1])]
    for call in calls:  # CPU tensors are refused before the library is reached
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        ea.kv4_cache(2, 2, 20, 128, device="cpu")
    with pytest.raises(AttributeError):
        ea.no_such_name


@pytest.mark.parametrize("page,d,other", [(128, 64, 128), (32, 64, 128), (64, 128, 64), (16, 128, 64)])
def test_a_cache_is_read_with_its_own_head_dim(page, d, other):
    """Both head dims divide its bytes: the other one would be read as pages of another size."""
    from exact_attention_13_gb300 import kv

    cache = ea.kv4_cache(3, 2, page, d, device="cpu")
    assert kv._cache_shape(cache, d) == (3, 2, page)
    with pytest.raises(ValueError, match=f"made for d = {d}"):
        kv._cache_shape(cache, other)
    assert kv._cache_shape(torch.empty_like(cache), d) == (3, 2, page)


def test_sizes_past_32_bits_are_refused_not_cut():
    from exact_attention_13_gb300 import kv

    for bad in ((2 ** 32 + 3, 2, 16, 64), (3, 2 ** 32 + 2, 16, 64), (3, 2, 2 ** 32 + 16, 64),
                (3, 2, 16, 2 ** 32 + 64), (-1, 2, 16, 64)):
        with pytest.raises(ValueError):
            ea.kv4_cache(*bad, device="meta")
    # sizes that the calls on a cache refuse: 2^31 slots, 65536 heads
    for bad in ((2 ** 27, 1, 16, 64), (2 ** 24, 1, 128, 128), (1, 65536, 16, 64)):
        assert ea.lib().fa_kv4_cache_bytes(*bad) == 0
        with pytest.raises(ValueError):
            ea.kv4_cache(*bad, device="meta")
    assert ea.kv4_cache(2 ** 27 - 1, 1, 16, 64, device="meta").shape == (2 ** 27 - 1, 1, 2, 16 * 36)
    assert ea.kv4_workspace_bytes(4, 2, 128, 1, 2 ** 32 + 64, 100) == 0
    assert ea.kv4_workspace_bytes(4, 2, 128, 1, 64, 2 ** 32 + 100) == 0
    assert ea.kv4_workspace_bytes(4, 2, 128, 2 ** 40, 64, 100) == ea.kv4_workspace_bytes(4, 2, 128, 2 ** 20, 64, 100)
    for shape in ((2 ** 31,), (1, 2 ** 32 + 4), (2, 2 ** 31)):
        wide = torch.empty(shape, dtype=torch.int32, device="meta")
        with pytest.raises(ValueError, match="2\\^31 - 1"):
            kv._ints(wide, shape, wide.get_device(), "table")
