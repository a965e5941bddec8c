"""Host-side checks of the paged-cache entry points that need no GPU: what include/fdma_paged.h declares is
exported, the packed argument bytes are the C structs, and bad arguments are refused before any CUDA call."""
import ctypes
import os
import re
import shutil
import struct

import pytest

from block_sparse_masked_02_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fdma_paged.h")


@pytest.fixture(scope="module")
def P():
    if not os.path.exists(B.LIB) and shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no nvcc to build libfdma")
    B.build()
    from block_sparse_masked_02_gb300 import paged

    return paged


def test_declared_entry_points_are_exported(P):
    declared = sorted(set(re.findall(r"FDMA_API\s+[\w\s\*]+?\b(fdma_\w+)\s*\(", open(HEADER).read())))
    assert declared == sorted(P.EXPORTED)
    lib = ctypes.CDLL(B.LIB)
    for name in declared:
        assert hasattr(lib, name), name


def test_packed_bytes_are_the_structs(P):
    c = list(range(1, 8)) + [11, 12, 13, 14, 21, 22, 23, 24, 31, 32, 33, 34, 41, 42, 43, 44, 51, 52, 53]
    got = P.FdmaKvCache.from_buffer_copy(P._PACK_CACHE(*c))
    assert (got.B, got.Hkv, got.d, got.cache_type, got.num_pages, got.page_size, got.max_pages) == tuple(range(1, 8))
    assert got.k == 11 and list(got.k_stride) == [12, 13, 14] and got.v == 21 and list(got.v_stride) == [22, 23, 24]
    assert got.k_exp == 31 and list(got.k_exp_stride) == [32, 33, 34]
    assert got.v_exp == 41 and list(got.v_exp_stride) == [42, 43, 44]
    assert (got.page_table, got.table_stride, got.k_len) == (51, 52, 53)
    a = P.FdmaPagedArgs.from_buffer_copy(P._PACK_ARGS(*c, 61, 62, 63, 64, 65, 66, 67, 1, 69, 70, 0.5, 72, 73))
    assert bytes(a.cache) == P._PACK_CACHE(*c)
    assert (a.T, a.Hq, a.q, list(a.q_stride), a.cu_q) == (61, 62, 63, [64, 65], 66)
    assert (a.max_q, a.causal, a.window, a.sinks, a.scale, a.workspace, a.workspace_bytes) == (67, 1, 69, 70, 0.5, 72, 73)
    assert len(P._PACK_ARGS(*c, *([0] * 10), 0.0, 0, 0)) == ctypes.sizeof(P.FdmaPagedArgs)
    assert bytes(a)[-16:] == P._PACK_WORKSPACE(72, 73)


FAKE = 1 << 20  # never dereferenced: the arguments are refused first


def _args(P, **kw):
    a = P.FdmaPagedArgs()
    c = a.cache
    c.B, c.Hkv, c.d, c.cache_type, c.num_pages, c.page_size, c.max_pages = 2, 2, 128, 0, 10, 16, 4
    c.k = c.v = c.k_exp = c.v_exp = c.page_table = c.k_len = FAKE
    c.k_stride[:] = c.v_stride[:] = [16 * 2 * 128, 2 * 128, 128]
    c.k_exp_stride[:] = c.v_exp_stride[:] = [32, 2, 1]
    c.table_stride = 4
    a.T, a.Hq, a.q, a.cu_q, a.max_q, a.causal, a.scale = 8, 4, FAKE, FAKE, 4, 1, 0.1
    a.q_stride[:] = [512, 128]
    for k, v in kw.items():
        if k.endswith("]"):
            name, i = k[:-1].split("[")
            getattr(c if hasattr(c, name) else a, name)[int(i)] = v
        else:
            setattr(c if hasattr(c, k) else a, k, v)
    return a


@pytest.mark.parametrize("field,value,status", [
    ("B", -1, 1), ("Hkv", 0, 1), ("Hq", 3, 1), ("Hq", 0, 1), ("d", 0, 1), ("d", 100, 2), ("d", 136, 2), ("cache_type", 2, 1),
    ("num_pages", -1, 1), ("page_size", 8, 2), ("page_size", 24, 2), ("page_size", 8192, 2), ("page_size", 0, 1),
    ("max_pages", -1, 1), ("max_pages", 1 << 27, 2), ("k", None, 1), ("v", FAKE + 8, 2), ("k_stride[1]", 4, 2),
    ("v_stride[0]", -8, 1), ("page_table", None, 1), ("k_len", None, 1), ("table_stride", -1, 1), ("T", -1, 1),
    ("max_q", -1, 1), ("causal", 2, 1), ("window", -1, 1), ("sinks", -1, 1), ("scale", 0.0, 1), ("scale", float("inf"), 1),
    ("scale", float("nan"), 1), ("q", None, 1), ("q", FAKE + 2, 2), ("q_stride[0]", 12, 2), ("q_stride[1]", -8, 1),
    ("cu_q", None, 1), ("T", 1 << 30, 2),
])
def test_attention_arguments_are_refused(P, field, value, status):
    a = _args(P, **{field: value})
    assert P.load().fdma_paged_fwd(bytes(a), FAKE, FAKE, None) == status


def test_attention_refuses_windows_without_causal_and_missing_buffers(P):
    lib = P.load()
    assert lib.fdma_paged_fwd(bytes(_args(P, window=8, causal=0)), FAKE, FAKE, None) == 1
    assert lib.fdma_paged_fwd(bytes(_args(P)), None, FAKE, None) == 1
    assert lib.fdma_paged_fwd(bytes(_args(P)), FAKE, None, None) == 1
    assert lib.fdma_paged_fwd(bytes(_args(P)), FAKE + 8, FAKE, None) == 2
    assert lib.fdma_paged_fwd(bytes(_args(P)), FAKE, FAKE, None) == 5  # no workspace
    need = lib.fdma_paged_workspace_size(bytes(_args(P)))
    a = _args(P, workspace=FAKE, workspace_bytes=need - 1)
    assert need > 0 and lib.fdma_paged_fwd(bytes(a), FAKE, FAKE, None) == 5
    assert lib.fdma_paged_fwd(bytes(_args(P, workspace=FAKE + 16, workspace_bytes=need)), FAKE, FAKE, None) == 5


def test_workspace_size_grows_with_the_rows_of_an_item_only(P):
    size = lambda **kw: P.load().fdma_paged_workspace_size(bytes(_args(P, **kw)))  # noqa: E731
    assert size(max_q=1) < size(max_q=8) < size(max_q=100) == size(max_q=100, max_pages=1 << 20) == size(max_q=5000)
    assert size(d=100) == 0 and size(Hq=3) == 0


@pytest.mark.parametrize("field,value,status", [
    ("d", 8, 2), ("d", 24, 2), ("k_exp", None, 1), ("k_exp_stride[2]", -1, 1), ("k_stride[2]", 8, 2), ("k_stride[0]", 0, 1),
    ("v_exp_stride[1]", 0, 1),
])
def test_quantised_caches_are_checked(P, field, value, status):
    a = _args(P, cache_type=1, **{field: value})
    st = struct.pack("2q", 256, 128)
    assert P.load().fdma_kv_append(bytes(a.cache), FAKE, st, FAKE, st, FAKE, 4, None) == status


def test_append_and_gather_arguments_are_refused(P):
    lib, c, st = P.load(), bytes(_args(P).cache), struct.pack("2q", 256, 128)
    assert lib.fdma_kv_append(c, None, st, FAKE, st, FAKE, 4, None) == 1
    assert lib.fdma_kv_append(c, FAKE, st, FAKE, st, None, 4, None) == 1
    assert lib.fdma_kv_append(c, FAKE, None, FAKE, st, FAKE, 4, None) == 1
    assert lib.fdma_kv_append(c, FAKE + 2, st, FAKE, st, FAKE, 4, None) == 2
    assert lib.fdma_kv_append(c, FAKE, struct.pack("2q", 257, 128), FAKE, st, FAKE, 4, None) == 2
    assert lib.fdma_kv_append(c, FAKE, st, FAKE, struct.pack("2q", 256, -8), FAKE, 4, None) == 1
    assert lib.fdma_kv_append(c, FAKE, st, FAKE, st, FAKE, -1, None) == 1
    assert lib.fdma_kv_append(c, FAKE, st, FAKE, st, FAKE, 0, None) == 0
    assert lib.fdma_kv_append(None, FAKE, st, FAKE, st, FAKE, 4, None) == 1
    assert lib.fdma_kv_gather(c, None, None, 4, FAKE, FAKE, None) == 1
    assert lib.fdma_kv_gather(c, FAKE, None, 4, None, FAKE, None) == 1
    assert lib.fdma_kv_gather(c, FAKE, None, 4, FAKE + 4, FAKE, None) == 2
    assert lib.fdma_kv_gather(c, FAKE, None, -4, FAKE, FAKE, None) == 1
    assert lib.fdma_kv_gather(c, FAKE, None, 0, None, None, None) == 0


def test_binding_refuses_cpu_tensors(P):
    import torch

    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens, cu = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: P.kv_append(k, k, kc, kc, table, lens, cu), lambda: P.kv_gather(kc, kc, table, lens, cu, 1),
                 lambda: P.fwd(k, kc, kc, table, lens, cu, 1)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
    with pytest.raises(ValueError):
        P.empty_cache(4, 16, 2, 64, dtype=torch.float16, device="cpu")
    kc, vc, ke, ve = P.empty_cache(4, 16, 2, 64, dtype=torch.float8_e4m3fn, device="cpu")
    assert kc.shape == (4, 16, 2, 64) and ke.shape == (4, 16, 2) and kc.stride(3) == 1 and kc.stride(1) == 64


def test_workspace_must_be_contiguous(P):
    torch = pytest.importorskip("torch")
    kc, vc, _, _ = P.empty_cache(4, 16, 2, 64, device="cpu")
    table, lens, cu = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([5], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    P.make_args(q, kc, vc, table, lens, cu, 1, workspace=torch.empty(64, dtype=torch.uint8))
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 30), torch.empty(64, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            P.make_args(q, kc, vc, table, lens, cu, 1, workspace=ws)


@pytest.mark.parametrize("field,value,status", [("scale", 3e38, 1), ("Hkv", (1 << 20) + 1, 2), ("B", (1 << 30) + 1, 2)])
def test_sizes_that_32_bit_arithmetic_does_not_hold_are_refused(P, field, value, status):
    """scale * log2(e) has to be finite in fp32; 2 * Hkv and B + 1 are formed in 32 bits."""
    kw = {field: value}
    if field == "Hkv":
        kw["Hq"] = value
    a = _args(P, **kw)
    lib, st = P.load(), struct.pack("2q", 256, 128)
    assert lib.fdma_paged_fwd(bytes(a), FAKE, FAKE, None) == status
    assert lib.fdma_paged_workspace_size(bytes(a)) == 0
    if field != "scale":
        assert lib.fdma_kv_append(bytes(a.cache), FAKE, st, FAKE, st, FAKE, 4, None) == status
        assert lib.fdma_kv_gather(bytes(a.cache), FAKE, None, 4, FAKE, FAKE, None) == status
