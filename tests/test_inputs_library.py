"""Host-side checks of the operators on attention's inputs that need no GPU: what include/fdma_inputs.h declares is
exported, the packed argument bytes are the C structs, and bad arguments are refused before any CUDA call."""
import ctypes
import os
import re
import shutil
import struct

import pytest

from block_sparse_masked_02_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fdma_inputs.h")
FAKE = 1 << 20  # never dereferenced: the arguments are refused first
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def I():  # noqa: E743
    if not os.path.exists(B.LIB) and shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no nvcc to build libfdma")
    B.build()
    from block_sparse_masked_02_gb300 import inputs

    return inputs


def test_declared_entry_points_are_exported(I):
    declared = sorted(set(re.findall(r"FDMA_API\s+[\w\s\*]+?\b(fdma_\w+)\s*\(", open(HEADER).read())))
    assert declared == sorted(I.EXPORTED)
    lib = ctypes.CDLL(B.LIB)
    for name in declared:
        assert hasattr(lib, name), name


def test_packed_bytes_are_the_structs(I):
    a = I.FdmaNormRopeArgs.from_buffer_copy(I._PACK_NORM_ROPE(1, 2, 3, 4, 5, 6, 0.5, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17, 18, 19, 20))
    assert (a.B, a.N, a.Hq, a.Hk, a.d, a.norm, a.eps, a.weight_type) == (1, 2, 3, 4, 5, 6, 0.5, 8)
    assert (a.q_weight, a.q_weight_head, a.k_weight, a.k_weight_head) == (9, 10, 11, 12)
    assert (a.rope, a.rope_len, a.rot, a.interleaved, a.first, a.positions, list(a.pos_stride)) == (13, 14, 15, 16, 17, 18, [19, 20])
    r = I.FdmaRows.from_buffer_copy(I._PACK_ROWS(1, 2, 3, 4))
    assert (r.p, list(r.stride)) == (1, [2, 3, 4])
    s = I.FdmaRelArgs.from_buffer_copy(I._PACK_REL(1, 2, 3, 4, 5, -6))
    assert (s.H, s.Nq, s.Nk, s.num_starts, s.two_sided, s.offset) == (1, 2, 3, 4, 5, -6)
    assert ctypes.sizeof(I.FdmaNormRopeArgs) == len(I._PACK_NORM_ROPE(*[0] * 6, 0.0, *[0] * 13))


def _args(I, **kw):
    a = I.FdmaNormRopeArgs()
    a.B, a.N, a.Hq, a.Hk, a.d, a.norm, a.eps = 2, 5, 4, 2, 128, 1, 1e-6
    a.q_weight = a.k_weight = a.rope = FAKE
    a.rope_len, a.rot = 10, 128
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _rows(I, p=FAKE, st=(2560, 512, 128)):
    return I._PACK_ROWS(p or 0, *st)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(Hq=0), 1), (dict(Hk=-1), 1), (dict(d=0), 1), (dict(d=100, rot=96), 2),
    (dict(d=264), 2), (dict(Hq=(1 << 20) + 1), 2), (dict(B=1 << 16, N=1 << 16), 2), (dict(norm=2), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(norm=0), 1),
    (dict(norm=0, q_weight=None, k_weight=None, rope=None, rot=0, rope_len=0), 1), (dict(weight_type=2), 1),
    (dict(Hk=0), 1), (dict(q_weight_head=-8), 1), (dict(q_weight_head=64), 1), (dict(q_weight=None, q_weight_head=128), 1),
    (dict(q_weight=FAKE + 4), 2), (dict(q_weight_head=132, k_weight_head=128), 2), (dict(q_weight_head=128), 2),
    (dict(interleaved=2), 1), (dict(rot=0), 1), (dict(rot=136), 1), (dict(rot=4), 2), (dict(rope=FAKE + 8), 2),
    (dict(rope=None), 1), (dict(rope=None, rot=0), 1), (dict(rope_len=-1), 1), (dict(first=-1), 1), (dict(first=6), 1),
    (dict(first=BIG), 1), (dict(rope_len=4), 1), (dict(positions=FAKE, pos_stride=(ctypes.c_int64 * 2)(-1, 1)), 1),
    (dict(positions=FAKE, pos_stride=(ctypes.c_int64 * 2)(0, -1)), 1),
])
def test_norm_rope_arguments_are_refused(I, kw, status):
    lib, a, r = I.load(), bytes(_args(I, **kw)), _rows(I)
    assert lib.fdma_norm_rope(a, r, r, r, r, None) == status
    assert lib.fdma_norm_rope_bwd(a, r, r, r, r, r, r, FAKE, FAKE, FAKE, 1 << 40, None) == status
    positions = any(k in kw for k in ("first", "positions")) or kw == dict(rope_len=4)
    assert (lib.fdma_norm_rope_bwd_workspace_size(a) == 0) != positions


@pytest.mark.parametrize("bad,status", [((None, (2560, 512, 128)), 1), ((FAKE + 8, (2560, 512, 128)), 2),
                                        ((FAKE, (2564, 512, 128)), 2), ((FAKE, (2560, 512, 124)), 2),
                                        ((FAKE, (2560, -512, 128)), 1)])
def test_rows_are_checked(I, bad, status):
    lib, a, r, x = I.load(), bytes(_args(I)), _rows(I), _rows(I, *bad)
    for i in range(4):
        t = [x if i == j else r for j in range(4)]
        assert lib.fdma_norm_rope(a, *t, None) == status
    for i in range(6):
        t = [x if i == j else r for j in range(6)]
        assert lib.fdma_norm_rope_bwd(a, *t, None, None, None, 0, None) == status


def test_rows_that_are_written_are_distinct(I):
    lib, a, r, same = I.load(), bytes(_args(I)), _rows(I), _rows(I, FAKE, (2560, 0, 128))
    assert lib.fdma_norm_rope(a, r, r, same, r, None) == 1
    assert lib.fdma_norm_rope(a, r, r, r, same, None) == 1
    assert lib.fdma_norm_rope_bwd(a, r, r, r, r, same, r, None, None, None, 0, None) == 1
    for st in ((2560, 512, 64), (2560, 448, 128), (2048, 512, 128), (0, 512, 128)):  # rows that overlap
        assert lib.fdma_norm_rope(a, r, r, _rows(I, FAKE, st), r, None) == 1, st
    assert lib.fdma_norm_rope(a, None, r, r, r, None) == 1
    assert lib.fdma_norm_rope(None, r, r, r, r, None) == 1


def test_weights_gradients_need_weights_and_a_workspace(I):
    lib, r = I.load(), _rows(I)
    a = bytes(_args(I, q_weight=None))
    assert lib.fdma_norm_rope_bwd(a, r, r, r, r, r, r, FAKE, None, FAKE, 1 << 40, None) == 1
    a = bytes(_args(I))
    need = lib.fdma_norm_rope_bwd_workspace_size(a)
    assert need > 0
    for ws, n in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert lib.fdma_norm_rope_bwd(a, r, r, r, r, r, r, FAKE, None, ws, n, None) == 5


def test_nothing_is_done_without_tokens(I):
    lib, r = I.load(), _rows(I)
    for kw in (dict(N=0, rope_len=0), dict(B=0)):
        a = bytes(_args(I, **kw))
        assert lib.fdma_norm_rope(a, None, None, None, None, None) == 0
        assert lib.fdma_norm_rope_bwd(a, r, r, r, r, r, r, None, None, None, 0, None) == 0
        assert lib.fdma_norm_rope_bwd_workspace_size(a) == 0


def _cache(P, **kw):
    c = P.FdmaKvCache()
    c.B, c.Hkv, c.d, c.cache_type, c.num_pages, c.page_size, c.max_pages = 2, 2, 128, 0, 10, 16, 4
    c.k = c.v = c.k_exp = c.v_exp = c.page_table = c.k_len = FAKE
    c.k_stride[:] = c.v_stride[:] = [16 * 2 * 128, 2 * 128, 128]
    c.k_exp_stride[:] = c.v_exp_stride[:] = [32, 2, 1]
    c.table_stride = 4
    for k, v in kw.items():
        setattr(c, k, v)
    return bytes(c)


def test_append_arguments_are_refused(I):
    from block_sparse_masked_02_gb300 import paged as P

    lib, r, c = I.load(), _rows(I), _cache(P)
    f, ok = lib.fdma_norm_rope_append, bytes(_args(I, B=1))
    for kw, status in ((dict(B=2), 1), (dict(B=1, Hk=1), 1), (dict(B=1, d=64, rot=64), 1), (dict(B=1, eps=0.0), 1),
                       (dict(B=1, N=-1), 1), (dict(B=1, positions=FAKE, pos_stride=(ctypes.c_int64 * 2)(0, -1)), 1)):
        assert f(bytes(_args(I, **kw)), c, r, r, r, r, FAKE, None) == status
    assert f(ok, None, r, r, r, r, FAKE, None) == 1
    assert f(None, c, r, r, r, r, FAKE, None) == 1
    assert f(ok, c, r, r, r, r, None, None) == 1
    for i in range(4):
        for bad, status in ((_rows(I, FAKE + 2), 2), (_rows(I, None), 1), (_rows(I, FAKE, (0, 516, 128)), 2), (None, 1)):
            assert f(ok, c, *[bad if i == j else r for j in range(4)], FAKE, None) == status
    assert f(ok, c, r, r, r, _rows(I, FAKE, (0, 0, 128)), FAKE, None) == 1
    for kw, status in ((dict(page_size=24), 2), (dict(k=None), 1), (dict(d=100), 2), (dict(cache_type=2), 1),
                       (dict(k_stride=(ctypes.c_int64 * 3)(0, 256, 128)), 1), (dict(cache_type=1, k_exp=None), 1)):
        assert f(ok, _cache(P, **kw), r, r, r, r, FAKE, None) == status
    assert f(bytes(_args(I, B=1, N=0)), c, None, None, None, None, None, None) == 0
    assert f(ok, _cache(P, B=0), None, None, None, None, None, None) == 0


STARTS = struct.pack("4i", 0, 1, 2, 4)


def _rel(I, **kw):
    a = I.FdmaRelArgs()
    a.H, a.Nq, a.Nk, a.num_starts, a.two_sided, a.offset = 2, 16, 24, 4, 0, 8
    for k, v in kw.items():
        setattr(a, k, v)
    return bytes(a)


@pytest.mark.parametrize("kw,status", [
    (dict(H=0), 1), (dict(Nq=-1), 1), (dict(Nk=-8), 1), (dict(num_starts=0), 1), (dict(two_sided=2), 1),
    (dict(offset=(1 << 30) + 1), 1), (dict(offset=-(1 << 30) - 1), 1), (dict(Nk=25), 2), (dict(Nq=131073), 2),
    (dict(Nk=131080), 2), (dict(H=(1 << 20) + 1), 2), (dict(num_starts=257), 2),
])
def test_bias_arguments_are_refused(I, kw, status):
    lib, two, three = I.load(), struct.pack("2q", 2, 1), struct.pack("2q", 384, 24)
    a = _rel(I, **kw)
    assert lib.fdma_rel_bias(a, STARTS, FAKE, 0, two, FAKE, three, None) == status
    assert lib.fdma_rel_bias_bwd(a, STARTS, 1, FAKE, struct.pack("3q", 768, 384, 24), 0, FAKE, FAKE, 1 << 40, None) == status
    assert lib.fdma_rel_bias_bwd_workspace_size(a, 1) == 0


def test_bias_buffers_are_checked(I):
    lib, a, ts = I.load(), _rel(I), struct.pack("2q", 2, 1)
    out = lambda h, r: struct.pack("2q", h, r)  # noqa: E731
    f = lambda a, *rest: lib.fdma_rel_bias(a, STARTS, *rest)  # noqa: E731
    for bad in (None, struct.pack("4i", 1, 2, 3, 4), struct.pack("4i", 0, 3, 2, 4)):
        assert lib.fdma_rel_bias(a, bad, FAKE, 0, ts, FAKE, out(384, 24), None) == 1
        assert lib.fdma_rel_bias_bwd(a, bad, 1, FAKE, struct.pack("3q", 768, 384, 24), 0, FAKE, FAKE, 1 << 40, None) == 1
    assert f(a, None, 0, ts, FAKE, out(384, 24), None) == 1
    assert f(a, FAKE, 2, ts, FAKE, out(384, 24), None) == 1
    assert f(a, FAKE, 0, struct.pack("2q", -1, 1), FAKE, out(384, 24), None) == 1
    assert f(a, FAKE, 0, ts, None, out(384, 24), None) == 1
    assert f(a, FAKE, 0, ts, FAKE + 8, out(384, 24), None) == 2
    for h, r, status in ((0, 24, 1), (384, 16, 1), (380, 24, 1), (384, 28, 1), (388, 24, 2), (392, 24, 0), (24, 48, 0), (24, 40, 1)):
        if status:  # (those that are allowed are not launched here)
            assert f(a, FAKE, 0, ts, FAKE, out(h, r), None) == status, (h, r)
    assert f(_rel(I, Nq=0), FAKE, 0, ts, None, out(0, 0), None) == 0
    assert f(_rel(I, Nk=0), FAKE, 0, ts, None, out(0, 0), None) == 0
    g = lambda a, *rest: lib.fdma_rel_bias_bwd(a, STARTS, *rest)  # noqa: E731
    ds = struct.pack("3q", 768, 384, 24)
    need = lib.fdma_rel_bias_bwd_workspace_size(a, 2)
    assert need > 0 and lib.fdma_rel_bias_bwd_workspace_size(a, 0) == 0 and lib.fdma_rel_bias_bwd_workspace_size(a, -1) == 0
    assert g(a, -1, FAKE, ds, 0, FAKE, FAKE, need, None) == 1
    assert g(a, 2, FAKE, ds, 2, FAKE, FAKE, need, None) == 1
    assert g(a, 2, None, ds, 0, FAKE, FAKE, need, None) == 1
    assert g(a, 2, FAKE, None, 0, FAKE, FAKE, need, None) == 1
    assert g(a, 2, FAKE, ds, 0, None, FAKE, need, None) == 1
    assert g(a, 2, FAKE + 8, ds, 0, FAKE, FAKE, need, None) == 2
    assert g(a, 2, FAKE, struct.pack("3q", 768, 388, 24), 0, FAKE, FAKE, need, None) == 2
    assert g(a, 2, FAKE, struct.pack("3q", 768, -384, 24), 0, FAKE, FAKE, need, None) == 1
    assert g(a, (1 << 20) + 1, FAKE, ds, 0, FAKE, FAKE, need, None) == 2
    for ws, n in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert g(a, 2, FAKE, ds, 0, FAKE, ws, n, None) == 5


def test_binding_refuses(I):
    import torch

    from block_sparse_masked_02_gb300 import paged as P

    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens, cu = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: I.norm_rope(x, x), lambda: I.norm_rope_bwd(x, x, x, x), lambda: I.rel_bias(torch.zeros(4, 2), 8, 8, (0, 1)),
                 lambda: I.rel_bias_bwd(torch.zeros(1, 2, 8, 8, dtype=torch.bfloat16), (0, 1)),
                 lambda: P.norm_rope_append(x, x, x, kc, kc, table, lens, cu)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
    w = torch.ones(64)
    good = (x, x, w, w, None, None, 0, False, True, 1e-6)
    I._norm_rope_args(*good)
    for i, bad in ((0, x[0]), (1, x[:, :, :32]), (2, w[:32]), (2, w.half()), (2, torch.ones(3, 64)), (2, torch.ones(128)[::2]),
                   (3, w.bfloat16()), (2, torch.ones(64).expand(2, 64)), (4, torch.zeros(4, 2, 32, dtype=torch.float64)),
                   (4, torch.zeros(4, 64)), (4, torch.zeros(4, 2, 64)[:, :, ::2]), (5, torch.zeros(1)),
                   (5, torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            I._norm_rope_args(*[bad if i == j else v for j, v in enumerate(good)])
    with pytest.raises(ValueError):
        I._norm_rope_args(x, None, None, w, None, None, 0, False, True, 1e-6)
    for bad in (x.float(), x[..., ::2], torch.zeros(2, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            I._rows("x", bad)
    with pytest.raises(ValueError):
        I._rows("x", x, x[:, :1].shape)
    for bad in ((1, 128), (3, 128), (32, 8), (33, 128)):
        with pytest.raises(ValueError):
            I.rel_starts(*bad)
    with pytest.raises(ValueError):
        I._rel_args(1, 8, 8, (), False, None)
    with pytest.raises(ValueError):
        I._rel_args(1, 8, 8, tuple(range(257)), False, None)


def test_workspaces_depend_on_sizes_alone(I):
    lib = I.load()
    size = lambda **kw: lib.fdma_norm_rope_bwd_workspace_size(bytes(_args(I, **kw)))  # noqa: E731
    assert size() == size(first=1, rope_len=11) == size(norm=1, rope=None, rot=0, rope_len=0)
    assert size(N=50000) < 2 ** 20 and size(q_weight_head=128, k_weight_head=128, N=50000) < 2 ** 23


def test_weights_gradients_that_are_not_wanted_are_not_taken(I):
    import torch

    x, w = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.ones(64)
    for grads in ((None, None, w, None), (None, None, None, w)):
        with pytest.raises(ValueError, match="want_dweight"):
            I.norm_rope_bwd(x, x, x, x, q_weight=w, k_weight=w, want_dweight=False, grads=grads)


def test_outputs_for_keys_without_keys_are_not_taken(I):
    import torch

    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="without keys"):
        I.norm_rope(x, k_out=x)
    with pytest.raises(ValueError, match="without keys"):
        I.norm_rope_bwd(x, None, x, None, grads=(None, x, None, None))


def test_a_weight_of_one_head_may_have_any_stride(I):
    import torch

    w = torch.ones(1, 129)[:, :128]
    assert I._weight("w", w, 1, 128) == (w.data_ptr(), 128, I.FDMA_FP32)
    w = w.as_strided((1, 128), (1, 1))
    assert I._weight("w", w, 1, 128) == (w.data_ptr(), 128, I.FDMA_FP32)
    w = torch.ones(2, 136)[:, :128]
    assert I._weight("w", w, 2, 128) == (w.data_ptr(), 136, I.FDMA_FP32)


def test_numbers_that_the_structs_do_not_hold_are_refused(I):
    import torch

    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for first, eps in ((1 << 31, 1e-6), (-(1 << 31) - 1, 1e-6), (0.5, 1e-6), (0, 1e39), (0, "1")):
        with pytest.raises(ValueError):
            I._norm_rope_args(x, None, None, None, None, None, first, False, True, eps)
    for starts, Nq, offset in (((0, 1 << 31), 8, None), ((0, 1.5), 8, None), ((0, 1), 8, 1 << 31), ((0, 1), 1 << 31, 0), ((0, 1), 8, 0.5)):
        with pytest.raises(ValueError):
            I._rel_args(1, Nq, 8, starts, False, offset)
