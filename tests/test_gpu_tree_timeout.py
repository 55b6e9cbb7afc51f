"""Attention of drafted trees gives up when a wait runs out: in a test build of the library whose copies (units of 32
and 64 rows) or widening warps (256 rows) deliver nothing, wait limit 50 ms, the call records FA_ERR_DEVICE_TIMEOUT in
the status word and ends, and the context stays usable."""
import ctypes
import os
import shutil
import subprocess
import time

import pytest

pytestmark = pytest.mark.gpu

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "exact_attention_13_gb300", "csrc")


@pytest.fixture(scope="module")
def stall(tmp_path_factory):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    path = str(tmp_path_factory.mktemp("stall") / "libexattn_tree_stall.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                    "--threads", "0", "-Xcompiler", "-fPIC", "-shared", "-DEXATTN_INJECT_STALL=1",
                    "-DEXATTN_WAIT_LIMIT_NS=50000000ull", "-o", path,
                    *(os.path.join(CSRC, f) for f in ("fa_api.cu", "kv_api.cu", "tree_api.cu"))], check=True)
    return ctypes.CDLL(path)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nodes,width", [(10, 20), (30, 20), (100, 20), (30, 2)])  # (two pages: units are not split)
def test_wait_timeout_sets_status_and_context_survives(stall, d, nodes, width):
    import torch

    import exact_attention_13_gb300 as ea

    stall.fa_kv4_tree_fwd.restype, stall.fa_kv4_tree_fwd.argtypes = ea.SIGNATURES["fa_kv4_tree_fwd"]
    B, page, Hq, Hkv = 3, 64, 4, 2
    n = min(1000, page * width)
    k = torch.randn(B * n, Hkv, d, device="cuda").bfloat16()
    cache = ea.kv4_cache(B * width, Hkv, page, d)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    at = torch.arange(n, device="cuda")
    slots = (table[:, at // page] * page + at % page).int().reshape(-1).contiguous()
    ea.kv4_append(k, k, cache, slots)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    off = torch.arange(0, (B + 1) * nodes, nodes, dtype=torch.int32, device="cuda")
    parents = torch.arange(-1, nodes - 1, dtype=torch.int32, device="cuda").repeat(B)
    seen = ea.tree_plan(parents, off, lens - nodes, nodes).seen
    q = torch.randn(B * nodes, Hq, d, device="cuda").bfloat16()
    want = ea.kv4_tree_fwd(q, cache, table, lens, off, seen, max_q=nodes)
    o, lse = torch.empty_like(q), torch.empty(B * nodes, Hq, device="cuda")
    size = ea.kv4_tree_workspace_bytes(Hq, Hkv, d, nodes, page, width)
    ws = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rc = stall.fa_kv4_tree_fwd(q.data_ptr(), Hq * d, d, cache.data_ptr(), B * width, page, table.data_ptr(), width,
                               lens.data_ptr(), off.data_ptr(), seen.data_ptr(), seen.shape[1], o.data_ptr(),
                               lse.data_ptr(), B * nodes, B, Hq, Hkv, d, nodes, 0.1, 1.0, 1.0, ws.data_ptr(), size,
                               status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == ea.FA_OK
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert int(status.item()) == ea.FA_ERR_DEVICE_TIMEOUT
    assert elapsed < 5.0, elapsed
    again = ea.kv4_tree_fwd(q, cache, table, lens, off, seen, max_q=nodes)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert ea.device_status(clear=True) == 0
