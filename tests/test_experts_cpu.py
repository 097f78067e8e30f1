"""Refusals of the expert operators, before any device is touched."""
import ctypes

import pytest

from neural_radiance_field_b200 import _capi
from neural_radiance_field_b200 import build as nbuild

BAD = _capi.NERF_ERR_INVALID_ARG
P = ctypes.c_void_p(4096)       # never dereferenced: validation fails first
ODD = ctypes.c_void_p(4097)     # aligned to no element
HALF = ctypes.c_void_p(4104)    # aligned to 8 bytes only


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return _capi.lib()


def refused(lib, why, status):
    assert status == BAD
    assert why in lib.nerf_last_error(None), lib.nerf_last_error(None)


def test_sort(lib):
    b = ctypes.c_int64()
    assert lib.nerf_expert_sort_workspace(786432, 8, 4096, ctypes.byref(b)) == 0 and 0 < b.value < 1 << 30
    for n, k, e, why in ((0, 8, 64, b"at least 1"), (4, 0, 64, b"at least 1"), (4, 65, 64, b"above 64"),
                         ((1 << 30) // 8 + 1, 8, 64, b"2^30 pairs"), (1 << 62, 64, 64, b"2^30 pairs"),
                         (4, 8, 0, b"1..4096"), (4, 8, 4097, b"1..4096")):
        refused(lib, why, lib.nerf_expert_sort_workspace(n, k, e, ctypes.byref(b)))
        refused(lib, why, lib.nerf_expert_sort(P, n, k, e, P, P, P, P, 1 << 40, None))
    refused(lib, b"NULL", lib.nerf_expert_sort_workspace(4, 8, 64, None))
    need = ctypes.c_int64()
    lib.nerf_expert_sort_workspace(1000, 8, 64, ctypes.byref(need))
    refused(lib, b"workspace too small", lib.nerf_expert_sort(P, 1000, 8, 64, P, P, P, P, need.value - 1, None))
    for args in ((None, P, P, P, P), (P, None, P, P, P), (P, P, P, None, P), (P, P, P, P, None)):
        refused(lib, b"NULL", lib.nerf_expert_sort(args[0], 4, 2, 8, args[1], args[2], args[3], args[4], 1 << 40, None))
    refused(lib, b"misaligned", lib.nerf_expert_sort(ODD, 4, 2, 8, P, P, P, P, 1 << 40, None))
    refused(lib, b"misaligned", lib.nerf_expert_sort(P, 4, 2, 8, P, P, P, HALF, 1 << 40, None))


def test_rows(lib):
    d, c = lib.nerf_expert_dispatch, lib.nerf_expert_combine
    db, cb = lib.nerf_expert_dispatch_backward, lib.nerf_expert_combine_backward

    def every(why, dtype=0, n=4, width=8, pos=P, k=2, w=None):
        refused(lib, why, d(P, dtype, n, width, pos, k, w, P, None))
        refused(lib, why, c(P, dtype, n, width, pos, k, w, P, None))
        refused(lib, why, db(P, P, dtype, n, width, pos, k, w, P, P, None))
        refused(lib, why, cb(P, P, dtype, n, width, pos, k, w, P, P, None))

    every(b"dtype", dtype=3)
    every(b"dtype", dtype=-1)
    every(b"at least 1", n=0)
    every(b"at least 1", k=0)
    every(b"above 64", k=65)
    every(b"2^30 pairs", n=1 << 30)
    every(b"width", width=0)
    every(b"width", width=(1 << 20) + 1)
    every(b"pos is NULL", pos=None)
    every(b"misaligned", pos=ODD)
    every(b"misaligned", w=ODD)
    refused(lib, b"NULL", d(None, 0, 4, 8, P, 2, None, P, None))
    refused(lib, b"NULL", d(P, 0, 4, 8, P, 2, None, None, None))
    refused(lib, b"NULL", c(None, 0, 4, 8, P, 2, None, P, None))
    refused(lib, b"misaligned", c(ODD, 1, 4, 8, P, 2, None, P, None))
    refused(lib, b"misaligned", d(P, 0, 4, 8, P, 2, None, ctypes.c_void_p(4098), None))
    refused(lib, b"d_rows is NULL", db(None, P, 0, 4, 8, P, 2, None, P, None, None))
    refused(lib, b"nothing to compute", db(P, P, 0, 4, 8, P, 2, None, None, None, None))
    refused(lib, b"needs x", db(P, None, 0, 4, 8, P, 2, None, P, P, None))
    refused(lib, b"d_out is NULL", cb(None, P, 0, 4, 8, P, 2, None, P, None, None))
    refused(lib, b"nothing to compute", cb(P, P, 0, 4, 8, P, 2, None, None, None, None))
    refused(lib, b"needs rows", cb(P, None, 0, 4, 8, P, 2, None, P, P, None))


def test_distill(lib):
    def call(student=P, dtype=0, n=4, e=64, tl=P, ti=P, k=8, t=1.0, scale=None, loss=P, grad=None):
        return lib.nerf_distill_topk(student, dtype, n, e, tl, ti, k, t, scale, loss, grad, None)
    for kw, why in ((dict(student=None), b"NULL"), (dict(tl=None), b"NULL"), (dict(ti=None), b"NULL"),
                    (dict(loss=None), b"NULL"), (dict(dtype=3), b"dtype"), (dict(n=0), b"n must"),
                    (dict(e=0), b"n_classes"), (dict(e=(1 << 30) + 1), b"n_classes"), (dict(k=0), b"k must"),
                    (dict(k=257), b"k must"), (dict(t=0.0), b"temperature"), (dict(t=-1.0), b"temperature"),
                    (dict(t=float("nan")), b"temperature"), (dict(t=float("inf")), b"temperature"),
                    (dict(t=1e-45), b"temperature"), (dict(t=3e-39), b"temperature"),
                    (dict(t=2.0 ** -61), b"temperature"), (dict(t=2.0 ** 61), b"temperature"),
                    (dict(t=3e38), b"temperature"), (dict(student=ODD, dtype=1), b"misaligned"),
                    (dict(grad=ctypes.c_void_p(4098)), b"misaligned"), (dict(scale=ODD), b"misaligned")):
        refused(lib, why, call(**kw))


def test_cells(lib):
    f, b = lib.nerf_cells_forward, lib.nerf_cells_backward
    need = ctypes.c_int64()
    assert lib.nerf_cells_backward_workspace(1000, 4096, ctypes.byref(need)) == 0 and need.value > 0
    for n, e, why in ((0, 8, b"n_rows"), ((1 << 30) + 1, 8, b"n_rows"), (8, 0, b"4096"), (8, 4097, b"4096")):
        refused(lib, why, lib.nerf_cells_backward_workspace(n, e, ctypes.byref(need)))
        refused(lib, why, f(P, P, n, P, e, P, P, None, None))
        refused(lib, why, b(P, P, n, P, e, P, P, P, P, P, 1 << 40, None))
    refused(lib, b"NULL", lib.nerf_cells_backward_workspace(8, 8, None))
    for args in ((None, P, P, P, P), (P, None, P, P, P), (P, P, None, P, P), (P, P, P, None, P), (P, P, P, P, None)):
        refused(lib, b"NULL", f(args[0], args[1], 8, args[2], 8, args[3], args[4], None, None))
    refused(lib, b"16-byte", f(P, P, 8, P, 8, P, HALF, None, None))
    refused(lib, b"16-byte", f(P, P, 8, P, 8, P, P, HALF, None))
    refused(lib, b"misaligned", f(ODD, P, 8, P, 8, P, P, None, None))
    for args in ((None, P, P, P), (P, None, P, P), (P, P, None, P), (P, P, P, None)):
        refused(lib, b"NULL", b(P, P, 8, P, 8, P, args[0], args[1], args[2], args[3], 1 << 40, None))
    refused(lib, b"16-byte", b(P, P, 8, P, 8, P, HALF, P, P, P, 1 << 40, None))
    lib.nerf_cells_backward_workspace(8, 8, ctypes.byref(need))
    refused(lib, b"workspace too small", b(P, P, 8, P, 8, P, P, P, P, P, need.value - 1, None))


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and devices of the tensors (CPU tensors here), before the library is called."""
    import torch
    import neural_radiance_field_b200 as nb
    ids, pos = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    x, rows = torch.zeros(4, 8), torch.zeros(8, 8)
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        nb.nerf_expert_dispatch(x, pos, rows)
    with pytest.raises(ValueError, match="CUDA"):
        nb.nerf_expert_sort(ids, 8, torch.zeros(9, dtype=i32), None, pos, torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        nb.nerf_expert_combine(rows.double(), pos, x)
    with pytest.raises(ValueError, match="2 dimensions"):
        nb.nerf_distill_topk(x, torch.zeros(4), torch.zeros(4, dtype=i32), 1.0, torch.zeros(4))
    with pytest.raises(ValueError, match="2 dimensions"):
        nb.nerf_cells_forward(x, x, pos, torch.zeros(3317), x)


def test_binding_refuses_sizes_that_would_be_cut_to_32_bits():
    """2^32 + 8 is not 8: tensors without memory, so that the refusal comes before anything else."""
    import torch
    import neural_radiance_field_b200 as nb
    big, i32 = (1 << 32) + 8, torch.int32
    meta = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="meta")  # noqa: E731
    wide, x = meta(4, big), meta(4, 8)
    ids, pos = meta(4, big, t=i32), meta(4, 2, t=i32)
    calls = [lambda: nb.nerf_expert_sort_workspace(4, 2, big), lambda: nb.nerf_expert_sort_workspace(4, big, 8),
             lambda: nb.nerf_expert_sort_workspace((1 << 64) + 4, 2, 8), lambda: nb.nerf_cells_backward_workspace(8, big),
             lambda: nb.nerf_cells_backward_workspace((1 << 64) + 8, 8),
             lambda: nb.nerf_expert_sort(pos, big, meta(big + 1, t=i32), None, pos, x),
             lambda: nb.nerf_expert_sort(ids, 8, meta(9, t=i32), None, ids, x),
             lambda: nb.nerf_expert_dispatch(wide, pos, wide), lambda: nb.nerf_expert_dispatch(x, ids, x),
             lambda: nb.nerf_expert_dispatch_backward(wide, None, pos, wide), lambda: nb.nerf_expert_dispatch_backward(x, x, ids, x),
             lambda: nb.nerf_expert_combine(wide, pos, wide), lambda: nb.nerf_expert_combine(x, ids, x),
             lambda: nb.nerf_expert_combine_backward(wide, None, pos, wide), lambda: nb.nerf_expert_combine_backward(x, x, ids, x),
             lambda: nb.nerf_distill_topk(wide, x, pos, 1.0, x), lambda: nb.nerf_distill_topk(x, x, ids, 1.0, x),
             lambda: nb.nerf_cells_forward(x, x, pos, meta(big, 3317), x),
             lambda: nb.nerf_cells_backward(x, x, pos, meta(big, 3317), x, x, x, x)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="fit (32|64) bits"):
            call()
            pytest.fail(f"call {i} was not refused")
