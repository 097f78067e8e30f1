"""The expert operators on the GPU against the fp64 oracle, within bounds derived
from the operations that each value goes through (u = 2^-24, the fp32 half step):
every bound below is a worst case, element by element."""
import numpy as np
import pytest

from nerf_inputs import kilonerf_weights
from oracle import experts as E

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ["fp32", "bf16", "fp16"]
HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -25}     # half a subnormal step at most


@pytest.fixture(scope="module")
def torch():
    import torch
    from neural_radiance_field_b200 import build
    build.build()
    return torch


def _t(torch, dtype):
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[dtype]


def _np(t):
    return t.detach().cpu().double().numpy()


def _cuda(torch, a, dtype=None):
    t = torch.from_numpy(np.array(a, order="C"))
    return t.cuda() if dtype is None else t.cuda().to(dtype)


def _near(got, ref, bound, name):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - ref)):.3e}, " \
                          f"at {np.argwhere(bad)[0]}: got {got[bad][0]!r}, want {ref[bad][0]!r}, bound {np.broadcast_to(bound, got.shape)[bad][0]:.3e}"


def _ids(rng, n, k, e, drop=0.15):
    """Distinct experts per point where there are enough, skewed; dropped pairs; some points all dropped."""
    ids = (e * rng.random((n, 1)) ** 2 + np.arange(k) * max(1, e // k)).astype(np.int64) % e
    ids[rng.random((n, k)) < drop] = -1
    ids[rng.random(n) < drop] = -1
    return ids.astype(np.int32)


def _sorted(torch, ids, e, order=True):
    import neural_radiance_field_b200 as nb
    n, k = ids.shape
    i32 = torch.int32
    off = torch.full((e + 1,), -7, device="cuda", dtype=i32)
    out = torch.full((n * k,), -7, device="cuda", dtype=i32) if order else None
    pos = torch.full((n, k), -7, device="cuda", dtype=i32)
    work = torch.empty(nb.nerf_expert_sort_workspace(n, k, e), device="cuda", dtype=torch.uint8)
    nb.nerf_expert_sort(ids, e, off, out, pos, work)
    return off, out, pos


# ------------------------------------------------------------------ sort

@pytest.mark.parametrize("n,k,e", [(1, 1, 1), (1, 8, 4096), (5, 3, 2), (31, 1, 7), (257, 2, 64), (1000, 8, 100),
                                   (4096, 2, 4096), (4099, 5, 1000), (20011, 8, 4096), (9973, 64, 33), (300001, 2, 3)])
@pytest.mark.parametrize("kind", ["mixed", "one expert", "all dropped"])
def test_sort(torch, n, k, e, kind):
    rng = np.random.default_rng([n, k, e])
    if kind == "mixed":
        ids = _ids(rng, n, k, e)
        ids[rng.random((n, k)) < 0.01] = e            # past the last expert: dropped too
        ids[rng.random((n, k)) < 0.01] = -(1 << 31)
    else:
        ids = np.full((n, k), e - 1 if kind == "one expert" else -1, np.int32)
    off, order, pos = _sorted(torch, _cuda(torch, ids), e)
    r_off, r_order, r_pos = E.sort(ids, e)
    m = r_order.size
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(pos.cpu().numpy(), r_pos)
    assert np.array_equal(order.cpu().numpy()[:m], r_order)
    assert (order.cpu().numpy()[m:] == -7).all()        # behind the last kept pair: as it was
    off2, _, pos2 = _sorted(torch, _cuda(torch, ids), e, order=False)
    assert torch.equal(off, off2) and torch.equal(pos, pos2)


@pytest.mark.parametrize("n,k,e", [(1300001, 8, 4096), (3700000, 8, 7), (2500, 2, 1025)])
def test_sort_of_many_tiles(torch, n, k, e):
    """Chunks of several tiles, three CTAs to an SM, and a chunk that ends inside a tile, against torch's sort."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = (e * torch.rand(n, k, generator=g, device="cuda") ** 3).int().clamp_(max=e - 1)
    ids[torch.rand(n, k, generator=g, device="cuda") < 0.05] = -1
    off, order, pos = _sorted(torch, ids, e)
    key = torch.where(ids < 0, e, ids).reshape(-1)
    by, ref = torch.sort(key, stable=True)
    m = int((by < e).sum())
    assert torch.equal(order[:m].long(), ref[:m]) and (order[m:] == -7).all()
    assert torch.equal(off.long(), torch.searchsorted(by, torch.arange(e + 1, device="cuda", dtype=by.dtype)))
    place = torch.empty_like(ref)
    place[ref] = torch.arange(n * k, device="cuda")
    assert torch.equal(pos.reshape(-1).long(), torch.where(key < e, place, -1))


@pytest.mark.parametrize("e", [5, 200, 4095, 4096])
@pytest.mark.parametrize("n", [777, 4096, 100003])
def test_sort_of_ids_that_meet_more_and_less(torch, n, e):
    """Runs of one expert, distinct ids, pairs of equal neighbours, ids that share a counter's word, dropped
    ones between them: stretches of each, so that a warp meets all of them in turn."""
    rng = np.random.default_rng([n, e])
    i = np.arange(n)
    kinds = np.stack([np.full(n, e - 1), i % e, (i // 2) % e, (i % 2) * ((e + 1) // 2) % e, (i // 16) % e, rng.integers(0, e, n),
                      rng.integers(0, min(e, 3), n), np.where(i % 3 == 0, -1, i % e), np.full(n, -1)])
    ids = kinds[rng.integers(0, len(kinds), n // 100 + 1)[i // 100], i].astype(np.int32).reshape(n, 1)
    off, order, pos = _sorted(torch, _cuda(torch, ids), e)
    r_off, r_order, r_pos = E.sort(ids, e)
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(pos.cpu().numpy(), r_pos)
    assert np.array_equal(order.cpu().numpy()[:r_order.size], r_order)


@pytest.mark.parametrize("n,k,e", [(60000, 2, 33), (60000, 2, 1000), (60000, 2, 4095)])
def test_sorts_back_to_back_share_a_workspace(torch, n, k, e):
    """Launch follows launch with other ids and one workspace, expert counts that no 32 divide."""
    import neural_radiance_field_b200 as nb
    rng = np.random.default_rng([n, k, e])
    all_ids = [_ids(rng, n, k, e, drop) for drop in (0.0, 0.3, 0.7)]
    ids = [_cuda(torch, i) for i in all_ids]
    work = torch.empty(nb.nerf_expert_sort_workspace(n, k, e), device="cuda", dtype=torch.uint8)
    outs = [(torch.empty(e + 1, device="cuda", dtype=torch.int32), torch.empty((n, k), device="cuda", dtype=torch.int32))
            for _ in range(60)]
    for r, (off, pos) in enumerate(outs):
        nb.nerf_expert_sort(ids[r % 3], e, off, None, pos, work)
    torch.cuda.synchronize()
    for r in range(3):
        off, _, pos = E.sort(all_ids[r], e)
        for got_off, got_pos in outs[r::3]:
            np.testing.assert_array_equal(got_off.cpu().numpy(), off)
            np.testing.assert_array_equal(got_pos.cpu().numpy(), pos)


@pytest.mark.parametrize("e", [2, 7, 1000, 4096])
@pytest.mark.parametrize("n", [3000, 200003])
def test_sort_of_two_experts_that_share_a_counter_word(torch, n, e):
    """Every 32 pairs meet in one word of two counters: what the lanes of one expert read of it comes before
    what a lane of either adds to it."""
    words = (e + 1) // 2
    low = np.random.default_rng([n, e]).integers(0, e - words, n // 500 + 1)[np.arange(n) // 500]
    ids = (low + words * np.random.default_rng([e, n]).integers(0, 2, n)).astype(np.int32).reshape(n, 1)
    off, order, pos = _sorted(torch, _cuda(torch, ids), e)
    r_off, r_order, r_pos = E.sort(ids, e)
    assert np.array_equal(off.cpu().numpy(), r_off)
    assert np.array_equal(pos.cpu().numpy(), r_pos)
    assert np.array_equal(order.cpu().numpy(), r_order)


def test_sort_agrees_with_the_cell_router(torch):
    """One cell per point: the same counts and cells as nerf_test_route_cells."""
    import neural_radiance_field_b200 as nb
    rng = np.random.default_rng(0)
    x = _cuda(torch, rng.uniform(-1.5, 1.4999, size=(5000, 3)).astype(np.float32))
    i32 = torch.int32
    cell = torch.empty(5000, device="cuda", dtype=i32)
    cnt, off = torch.empty(4096, device="cuda", dtype=i32), torch.empty(4097, device="cuda", dtype=i32)
    order = torch.empty(5000, device="cuda", dtype=i32)
    nb.nerf_test_route_cells(x, cell, cnt, off, order)
    mine, my_order, _ = _sorted(torch, cell[:, None].contiguous(), 4096)
    assert torch.equal(mine, off)
    assert torch.equal(cell[my_order.long()], cell[order.long()])


# ------------------------------------------------------------------ rows

def _rows_case(torch, rng, n, k, e, width, dtype, weighted, shift=0):
    """Inputs on the device and, as read back from it, in fp64; `shift` elements off the 16-byte boundary."""
    ids = _ids(rng, n, k, e)
    pos = E.sort(ids, e)[2]
    t = _t(torch, dtype)

    def make(m):
        flat = torch.empty(m * width + shift, device="cuda", dtype=t)
        flat.copy_(_cuda(torch, rng.normal(size=m * width + shift)))
        return flat[shift:].view(m, width)

    w = rng.normal(size=(n, k)).astype(np.float32) if weighted else None
    if weighted:
        w[pos < 0] = np.nan                            # what lies in a dropped place is not looked at
    return pos, _cuda(torch, pos.astype(np.int32)), w, None if w is None else _cuda(torch, w), make


ROWS = [(1, 1, 1, 1), (1, 8, 4096, 4), (3, 2, 5, 3), (193, 2, 64, 63), (300, 8, 4096, 4), (257, 3, 17, 27), (64, 4, 8, 256),
        (50, 2, 8, 1024), (100, 9, 16, 32), (33, 64, 100, 6), (20, 2, 4, 1023), (7, 12, 20, 2050), (40, 1, 3, 90)]


@pytest.mark.parametrize("n,k,e,width", ROWS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weighted,shift", [(True, 0), (False, 0), (True, 1), (True, 2)])
def test_rows(torch, n, k, e, width, dtype, weighted, shift):
    import neural_radiance_field_b200 as nb
    rng = np.random.default_rng([n, k, e, width, TYPES.index(dtype), weighted, shift])
    pos, pos_t, w, w_t, make = _rows_case(torch, rng, n, k, e, width, dtype, weighted, shift)
    hs, tiny = HALF_STEP[dtype], TINY[dtype]
    aw = np.where(pos >= 0, np.abs(w.astype(np.float64)) if weighted else 1.0, 0.0)
    x, rows, old = make(n), make(n * k), make(n * k)
    # dispatch: one product, rounded once to fp32 and once to the type; untouched rows keep their bits
    got = old.clone() if shift == 0 else old
    before = _np(got)
    nb.nerf_expert_dispatch(x, pos_t, got, w_t)
    ref = E.dispatch(_np(x), pos, w, before)
    exact = np.ones(n * k, bool)
    exact[pos[pos >= 0]] = not weighted
    assert np.array_equal(_np(got)[exact], ref[exact])
    _near(_np(got), ref, (U + hs + U * hs) * np.abs(ref) + tiny, "rows")
    # combine: k fused steps in fp32 (each within u of the running sum), one rounding
    out = make(n)
    nb.nerf_expert_combine(rows, pos_t, out, w_t)
    ref = E.combine(_np(rows), pos, w)
    mag = (aw[..., None] * np.abs(E.taken(_np(rows), pos))).sum(1)
    _near(_np(out), ref, hs * np.abs(ref) + (1 + hs) * 1.01 * k * U * mag + tiny, "out")
    assert (_np(out)[(pos < 0).all(1)] == 0).all()
    # their gradients; a dot product of `width` terms in any order: width * u of the sum of magnitudes
    d_x, dw = make(n), torch.full((n, k), 7.0, device="cuda")
    nb.nerf_expert_dispatch_backward(rows, x, pos_t, d_x, w_t, dw)
    assert torch.equal(d_x, out)                       # the same sum as combine, whether or not d_weights is asked for
    r_dw = E.dots(_np(rows), _np(x), pos)
    b_dw = 1.01 * (width + 1) * U * (np.abs(E.taken(_np(rows), pos)) * np.abs(_np(x))[:, None]).sum(2) + TINY["fp32"]
    _near(_np(dw), r_dw, b_dw, "d_weights")
    assert (_np(dw)[pos < 0] == 0).all()
    d_rows, dw2 = old.clone(), torch.full((n, k), 7.0, device="cuda")
    d_rows.copy_(_cuda(torch, before))
    if shift:
        d_rows = make(n * k)
        d_rows.copy_(_cuda(torch, before))
    nb.nerf_expert_combine_backward(x, rows, pos_t, d_rows, w_t, dw2)
    assert torch.equal(d_rows, got)                    # the same products as dispatch
    _near(_np(dw2), r_dw, b_dw, "d_weights of combine")
    # either output alone is the same
    only = torch.full((n, k), 7.0, device="cuda")
    nb.nerf_expert_dispatch_backward(rows, x, pos_t, None, w_t, only)
    assert torch.equal(only, dw)
    nb.nerf_expert_combine_backward(x, rows, pos_t, None, w_t, only)
    assert torch.equal(only, dw2)
    d_x2 = make(n)
    nb.nerf_expert_dispatch_backward(rows, None, pos_t, d_x2, w_t, None)
    assert torch.equal(d_x2, d_x)


@pytest.mark.parametrize("k", [1, 3, 8, 12])
@pytest.mark.parametrize("width,shift", [(1 << 20, 0), (1 << 20, 1), (70001, 0), (4096, 0), (4100, 0), (8191, 1), (8224, 0)])
@pytest.mark.parametrize("dtype", TYPES)
def test_weight_gradients_of_wide_rows(torch, width, shift, k, dtype):
    """Equal terms, whose roundings all go one way, and terms of one sign: eight lanes sum runs of 512 terms, then the
    runs in order, then each other, so no sum has more than 512 + width / 4096 + 4 roundings."""
    import neural_radiance_field_b200 as nb
    gen = torch.Generator(device="cuda").manual_seed(width + k)
    n, t = 2, _t(torch, dtype)

    def make(m):
        flat = torch.rand(m * width + shift, device="cuda", generator=gen).to(t)
        flat[:m * width // 2] = 0.1
        return flat[shift:].view(m, width)

    x, rows, d_x = make(n), make(n * k), make(n)
    pos = torch.randperm(n * k, device="cuda", generator=gen).int().view(n, k)
    pos[1, k - 1] = -1
    dw, dw2 = torch.full((n, k), 7.0, device="cuda"), torch.full((n, k), 7.0, device="cuda")
    nb.nerf_expert_dispatch_backward(rows, x, pos, d_x, None, dw)
    ref = E.dots(_np(rows), _np(x), pos.cpu().numpy())
    bound = (512 + width / 4096 + 4) * U * ref
    _near(_np(dw), ref, bound, "dispatch")
    nb.nerf_expert_combine_backward(x, rows, pos, torch.empty(n * k * width + shift, device="cuda", dtype=t)[shift:].view(n * k, width), None, dw2)
    _near(_np(dw2), ref, bound, "combine")
    out = torch.empty_like(d_x) if shift == 0 else make(n)
    nb.nerf_expert_combine(rows, pos, out)
    assert torch.equal(out, d_x)                         # the sum does not depend on whether d_weights is asked for


def test_rows_nonfinite(torch):
    """An infinity or NaN in a kept row reaches its own point only; in rows that nothing names it reaches none."""
    import neural_radiance_field_b200 as nb
    pos = torch.tensor([[0, 1], [2, -1], [-1, -1]], device="cuda", dtype=torch.int32)
    for width in (4, 5, 64):
        for dtype in TYPES:
            rows = torch.ones(6, width, device="cuda", dtype=_t(torch, dtype))
            rows[3:] = float("nan")
            rows[1, 2] = float("inf")
            out = torch.empty(3, width, device="cuda", dtype=rows.dtype)
            nb.nerf_expert_combine(rows, pos, out, torch.full((3, 2), 2.0, device="cuda"))
            ref = torch.full((3, width), 2.0, device="cuda")
            ref[0] = 4.0
            ref[0, 2] = float("inf")
            ref[2] = 0.0
            assert torch.equal(out.float(), ref)


def test_rows_positions_out_of_range_are_dropped(torch):
    import neural_radiance_field_b200 as nb
    pos = torch.tensor([[0, 4], [1 << 30, -(1 << 31)]], device="cuda", dtype=torch.int32)   # n * k = 4 rows
    rows = torch.zeros(4, 8, device="cuda")
    nb.nerf_expert_dispatch(torch.ones(2, 8, device="cuda"), pos, rows)
    assert rows[0].eq(1).all() and rows[1:].eq(0).all()
    out = torch.empty(2, 8, device="cuda")
    nb.nerf_expert_combine(torch.full((4, 8), 3.0, device="cuda"), pos, out)
    assert out[0].eq(3).all() and out[1].eq(0).all()


# ------------------------------------------------------------------ distillation

def _distill_bounds(s, teacher, ids, T, scale, loss, grad, k):
    """Worst-case error of (loss, grad in fp32). The exponent's argument (s - m) / T: the difference, the
    factor (two roundings) and the product, 4u |z - m| <= 8uA with z = s / T and A = max |z|; an exponential
    within 2^-22 (4u), with 2u for a rescaled running sum. A sum of the classes in at most classes / 32 + 16
    steps. log within 2 steps of its value."""
    z = s / T
    n, e = s.shape
    fin = np.where(np.isfinite(z), np.abs(z), 0.0)
    A = fin.max(1)
    d_exp = U * (8 * A + 6)
    d_sum = d_exp + U * (e / 32 + 16)
    lz = np.log(e) + 2 * A
    d_logq = U * (4 * A + 2 * A) + d_sum + 4 * U * lz + 3 * U * (2 * A + lz)
    kept = (ids >= 0) & (ids < e) & (teacher != -np.inf)
    tz = np.where(kept, teacher / T, 0.0)
    At = np.abs(tz).max(1)
    d_p = U * (2 * (6 * At + 4) + k + 4)
    d_logp = U * (4 * At + 2 * At) + U * (6 * At + 4 + k) + 8 * U * np.log(k + 1) + 3 * U * (2 * At + np.log(k + 1))
    big = 2 * At + 2 * A + np.log(k + 1) + lz                      # |log p - log q| of a kept class
    b_loss = 1.01 * T * T * (d_logq + d_logp + (d_p + U * (k + 4)) * big)
    q = np.where(np.isfinite(z), np.exp(z - z.max(1, keepdims=True)), 0.0)
    q /= q.sum(1, keepdims=True)
    p = np.zeros((n, e))
    for i in range(n):
        if kept[i].any():
            y = np.exp(tz[i][kept[i]] - tz[i][kept[i]].max())
            np.add.at(p[i], ids[i][kept[i]], y / y.sum())
    b_grad = 1.01 * np.abs(scale * T)[:, None] * (q * (d_exp + d_sum + 4 * U)[:, None] + p * (d_p + U * (k + 2))[:, None]
                                                 + U * (q + p)) + 3 * U * np.abs(grad)
    return b_loss, b_grad


DISTILL = [(1, 1, 1), (1, 8, 4096), (5, 3, 2), (33, 8, 31), (64, 16, 100), (17, 5, 333), (9, 32, 1024), (20, 16, 4096),
           (1300, 8, 4096), (1201, 3, 1501), (7, 256, 5000), (6, 9, 8191), (4, 32, 20001), (3, 40, 100003), (2, 7, 262144), (300, 2, 64)]


@pytest.mark.parametrize("n,k,e", DISTILL)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_distill(torch, n, k, e, dtype, shift):
    import neural_radiance_field_b200 as nb
    rng = np.random.default_rng([n, k, e, TYPES.index(dtype)])
    T = 1.5
    t = _t(torch, dtype)
    base = torch.empty(n * e + shift, device="cuda", dtype=t)
    base.copy_(_cuda(torch, 2.5 * rng.normal(size=n * e + shift)))
    student = base[shift:].view(n, e)
    ids = np.stack([rng.choice(e, size=k, replace=e < k) for _ in range(n)]).astype(np.int32)
    teacher = (3 * rng.normal(size=(n, k))).astype(np.float32)
    if n > 1:
        ids[rng.random((n, k)) < 0.2] = -1
        ids[n // 2] = -1                               # a row that keeps nothing
    if n > 2:
        teacher[1, 0] = -np.inf                        # a kept place whose logit is masked
        teacher[2] = -np.inf                           # a row whose logits all are
        ids[0, 0] = ids[0, -1] = e - 1                 # an id twice (k = 1: once)
        ids[3 % n, k // 2] = e                         # past the last class
        masked = np.setdiff1d(rng.choice(e, size=e // 3, replace=False), ids[0])
        student[0, _cuda(torch, masked)] = float("-inf")
    scale = rng.random(n).astype(np.float32) + 0.5
    args = (_cuda(torch, teacher), _cuda(torch, ids), T)
    loss = torch.full((n,), 7.0, device="cuda")
    gbase = torch.full((n * e + shift,), 7.0, device="cuda", dtype=t)
    grad = gbase[shift:].view(n, e)
    nb.nerf_distill_topk(student, *args, loss, grad, _cuda(torch, scale))
    r_loss, r_grad = E.distill(_np(student), teacher.astype(np.float64), ids, T, scale)
    b_loss, b_grad = _distill_bounds(_np(student), teacher.astype(np.float64), ids, T, scale.astype(np.float64), r_loss, r_grad, k)
    _near(_np(loss), r_loss, b_loss, "loss")
    hs = HALF_STEP[dtype]
    _near(_np(grad), r_grad, (1 + hs) * b_grad + hs * np.abs(r_grad) + TINY[dtype], "grad")
    if n > 2:
        assert loss[2] == 0 and grad[2].eq(0).all()
    if n > 1:
        assert loss[n // 2] == 0 and grad[n // 2].eq(0).all()
    if shift:
        assert gbase[0] == 7.0
    alone = torch.full((n,), 7.0, device="cuda")
    nb.nerf_distill_topk(student, *args, alone)
    assert torch.equal(alone, loss)
    other = torch.empty(n * e + 2, device="cuda", dtype=t)[2:].view(n, e)      # aligned unlike the student: same bounds
    nb.nerf_distill_topk(student, *args, alone, other, _cuda(torch, scale))
    _near(_np(alone), r_loss, b_loss, "loss, unlike alignment")
    _near(_np(other), r_grad, (1 + hs) * b_grad + hs * np.abs(r_grad) + TINY[dtype], "grad, unlike alignment")
    ones = torch.empty_like(gbase)[shift:].view(n, e)
    nb.nerf_distill_topk(student, *args, alone, ones)
    nb.nerf_distill_topk(student, *args, alone, grad, torch.ones(n, device="cuda"))
    assert torch.equal(ones, grad)


@pytest.mark.parametrize("e", [40, 4096, 20001, 120001])
def test_distill_temperatures_at_the_ends(torch, e):
    """The lowest and the highest temperature that the call takes."""
    import neural_radiance_field_b200 as nb
    rng = np.random.default_rng(e)
    n, k = 5, 6
    s = np.stack([rng.permutation(e) for _ in range(n)]).astype(np.float32)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(n)]).astype(np.int32)
    teacher = np.stack([rng.permutation(k) for _ in range(n)]).astype(np.float32)
    loss, grad = torch.empty(n, device="cuda"), torch.empty(n, e, device="cuda")
    T = 2.0 ** -60                                      # both distributions are one class: loss T (max s - s of the teacher's)
    nb.nerf_distill_topk(_cuda(torch, s), _cuda(torch, teacher), _cuda(torch, ids), T, loss, grad)
    want, rows = np.zeros((n, e)), np.arange(n)
    want[rows, s.argmax(1)] += T
    best = ids[rows, teacher.argmax(1)]
    want[rows, best] -= T
    assert np.array_equal(_np(grad), want)
    gap = T * (s.max(1) - s[rows, best]).astype(np.float64)
    _near(_np(loss), gap, 8 * U * gap, "loss")          # 1 / T, T T and powers of two are exact; the sums add zeros
    T, one = 2.0 ** 60, np.ones(n)
    nb.nerf_distill_topk(_cuda(torch, s), _cuda(torch, teacher), _cuda(torch, ids), T, loss, grad)
    r_loss, r_grad = E.distill(s, teacher, ids, T)
    b_loss, b_grad = _distill_bounds(s.astype(np.float64), teacher.astype(np.float64), ids, T, one, r_loss, r_grad, k)
    _near(_np(loss), r_loss, b_loss, "loss")
    _near(_np(grad), r_grad, b_grad + U * np.abs(r_grad), "grad")


@pytest.mark.parametrize("e", [40, 4096, 20001])
def test_distill_masks_and_extremes(torch, e):
    """Masks of the lowest value and of -inf, a kept class that the student rules out, NaN in rows that
    keep nothing, and rows beside each other that must not mix."""
    import neural_radiance_field_b200 as nb
    low = torch.finfo(torch.float32).min
    s = torch.zeros(6, e, device="cuda")
    s[5] = low                                          # every class masked by it: all alike
    s[0, 1:] = low                                      # all mass on class 0
    s[1, 1:] = float("-inf")
    s[2] = float("nan")
    s[3, 0] = float("-inf")                            # the teacher's only class is ruled out
    ids = torch.tensor([[0, -1], [0, -1], [-1, -1], [0, -1], [1, 2], [1, 2]], device="cuda", dtype=torch.int32)
    tl = torch.zeros(6, 2, device="cuda")
    tl[5] = low                                         # the teacher's entries too
    loss, grad = torch.empty(6, device="cuda"), torch.empty(6, e, device="cuda")
    nb.nerf_distill_topk(s, tl, ids, 0.5, loss, grad)   # 1 / T > 1: the lowest value times it overflows
    assert loss[5] == loss[4] and torch.equal(grad[5], grad[4])
    nb.nerf_distill_topk(s, tl, ids, 1.0, loss, grad)
    assert loss[5] == loss[4] and torch.equal(grad[5], grad[4])
    assert loss[:3].eq(0).all() and grad[:3].eq(0).all()
    assert loss[3] == float("inf") and torch.isfinite(grad[3]).all() and grad[3, 0] == -1
    want = np.log(e) - np.log(2)
    assert abs(loss[4].item() - want) <= 20 * U * (np.log(e) + 2) + (e / 32 + 16) * U


@pytest.mark.parametrize("e", [40, 4096, 20001, 300000])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0.125, 0.5, 1.0])
def test_distill_classes_kept_by_the_teacher_and_masked_by_the_student(torch, e, dtype, T):
    """The student's lowest value at a class that the teacher keeps: T^2 p (log p - log q) is T p |lowest| and some,
    finite although lowest / T may not be. The gap, its product with p, the sum of at most 3 and the product with T:
    6u of it; p within 2u (2 * 2 + k + 4), as in _distill_bounds with logits of at most 1 / T; the rest of the loss
    is below half a step of it in fp32 and bf16 and has the bound of T^2 (log e + 2) (e / 32 + 64) u in fp16."""
    import neural_radiance_field_b200 as nb
    low = torch.finfo(_t(torch, dtype)).min
    s = torch.zeros(4, e, device="cuda", dtype=_t(torch, dtype))
    s[:, 5] = 2.0
    s[:, 1] = low
    s[1, 7:] = low
    ids = torch.tensor([[1, -1, -1], [1, 5, -1], [2, 1, 5], [0, 5, 3]], device="cuda", dtype=torch.int32)
    tl = torch.tensor([[1.0, 0, 0], [0.5, 1, 0], [0, 1, 0.25], [0, 1, 0.5]], device="cuda")
    shifted = torch.empty(4 * e + 1, device="cuda", dtype=s.dtype)[1:].view(4, e)      # gradient aligned unlike the student
    for grad in (None, torch.empty_like(s), shifted):
        loss = torch.empty(4, device="cuda")
        nb.nerf_distill_topk(s, tl, ids, T, loss, grad)
        ref, r_grad = E.distill(_np(s), _np(tl), ids.cpu().numpy(), T)
        assert np.isfinite(ref.astype(np.float32)).all()
        bound = ref * U * (6 + 2 * (6 / T + 4) + 7) + T * T * (np.log(e) + 2 + 4 / T) * (e / 32 + 64) * U
        _near(_np(loss), ref, bound, "loss")
        if grad is not None:
            assert torch.isfinite(grad).all() and grad[0, 1] == -T and abs(r_grad[0, 1] + T) < 1e-9


@pytest.mark.parametrize("e,dtype", [(5003, "fp32"), (20001, "fp32"), (60000, "bf16"), (100003, "fp32")])
def test_distill_rows_of_one_call_are_those_of_calls_of_their_own(torch, e, dtype):
    """A CTA, and clusters of two, four and eight, that take several rows one after another: each row's loss and
    gradient are the bits of a call on it alone."""
    import neural_radiance_field_b200 as nb
    gen = torch.Generator(device="cuda").manual_seed(e)
    n, k, t = 700, 5, _t(torch, dtype)
    s = torch.randn(n, e, device="cuda", generator=gen).to(t)
    tl, ti = torch.randn(n, k, device="cuda", generator=gen), torch.randint(0, e, (n, k), device="cuda", generator=gen, dtype=torch.int32)
    ti[::7] = -1
    loss, grad = torch.full((n,), 7.0, device="cuda"), torch.full((n, e), 7.0, device="cuda", dtype=t)
    nb.nerf_distill_topk(s, tl, ti, 2.0, loss, grad)
    for i in (0, 1, 6, 7, 36, 37, 147, 148, 295, 296, 297, 443, 592, 699):
        one, g = torch.empty(1, device="cuda"), torch.empty(n, e, device="cuda", dtype=t)[i:i + 1]   # aligned like row i
        nb.nerf_distill_topk(s[i:i + 1], tl[i:i + 1], ti[i:i + 1], 2.0, one, g)
        assert torch.equal(one[0], loss[i]) and torch.equal(g[0], grad[i])


# ------------------------------------------------------------------ per-cell networks

C3 = 1.25 * 2.0 ** -20      # a product of two operands split in three: lo parts read at 2^-10, lo * lo dropped


def _encoding_errors(x, d):
    """Bound on the encodings' errors. An even octave's sine and cosine are within e = 2 steps (2^-23) of
    the angle's; the odd octave above it comes by doubling, 2sc and 1 - 2s^2, whose errors are at most
    2 (|s| + |c|) e and 4 |s| e (both <= 4e) and one rounding (2^-24). The unit direction's coordinates are
    within 3.5u of their value, times the angle's slope."""
    value = np.tile(np.where(np.arange(2) == 0, 1.0, 4.5) * 2.0 ** -23, 15)        # octaves 0, 1, 0, 1, ..
    ex = np.concatenate([np.zeros((len(x), 3)), np.tile(value, (len(x), 2))], axis=1)
    u = np.abs(d / np.linalg.norm(d, axis=1, keepdims=True))
    slope = np.pi * 2.0 ** np.arange(4)
    ang = (u[:, :, None] * slope).reshape(len(d), 12) * 3.5 * U + value[:12]
    return ex, np.concatenate([u * 3.5 * U, ang, ang], axis=1)


def _cells_case(torch, seed, counts, extra=0):
    rng = np.random.default_rng(seed)
    offset = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(offset[-1]) + extra
    x = rng.uniform(-1.5, 1.5, size=(max(n, 1), 3)).astype(np.float32)
    d = (rng.normal(size=(max(n, 1), 3)) * 3).astype(np.float32)
    return rng, offset, x, d, kilonerf_weights(seed, n_cells=len(counts))


COUNTS = {"one row": [1], "a tile less one": [0, 127], "a tile": [128, 0, 0], "a tile and one": [129, 3],
          "ragged": [0, 1, 7, 64, 130, 0, 300, 31, 128, 257, 0], "no rows": [0, 0], "many small": [3] * 700,
          "a hot cell": [5, 4000, 0, 2] + [1] * 30}


@pytest.mark.parametrize("name", list(COUNTS))
def test_cells(torch, name):
    import neural_radiance_field_b200 as nb
    counts = COUNTS[name]
    rng, offset, x, d, w = _cells_case(torch, len(counts), counts, extra=5)
    n, m = len(x), int(offset[-1])
    xt, dt, ot, wt = (_cuda(torch, a) for a in (x, d, offset, w))
    raw, hid = torch.full((n, 4), 7.0, device="cuda"), torch.full((n, 64), 7.0, device="cuda")
    nb.nerf_cells_forward(xt, dt, ot, wt, raw, hid)
    r_raw, r_hid = E.cells_forward(x, d, offset, w)
    px, pd = E.encodings(x, d)
    ex, ed = _encoding_errors(x, d.astype(np.float64))
    b_raw, b_hid = np.zeros((n, 4)), np.zeros((n, 64))
    for c in range(len(counts)):
        r = slice(offset[c], offset[c + 1])
        w1, b1, w2, b2, ws, bs, wc, bc = (np.abs(v) for v in E.cell_parts(w[c]))
        h1, h2 = r_hid[r, :32], r_hid[r, 32:]
        e1 = ex[r] @ w1.T + (C3 + 66 * U) * (np.abs(px[r]) @ w1.T + b1)
        e2 = e1 @ w2.T + (C3 + 35 * U) * ((h1 + e1) @ w2.T + b2)
        b_hid[r] = np.concatenate([e1, e2], axis=1)
        both, eb = np.concatenate([h2, np.abs(pd[r])], axis=1), np.concatenate([e2, ed[r]], axis=1)
        b_raw[r, :3] = eb @ wc.T + (C3 + 62 * U) * ((both + eb) @ wc.T + bc)
        b_raw[r, 3] = e2 @ ws + (C3 + 35 * U) * ((h2 + e2) @ ws + bs)
    _near(_np(hid)[:m], r_hid[:m], 1.01 * b_hid[:m] + 1e-30, "hidden")
    _near(_np(raw)[:m], r_raw[:m], 1.01 * b_raw[:m] + 1e-30, "raw")
    assert raw[m:].eq(7.0).all() and hid[m:].eq(7.0).all()       # rows behind the last: as they were
    raw2 = torch.full((n, 4), 7.0, device="cuda")
    nb.nerf_cells_forward(xt, dt, ot, wt, raw2)
    assert torch.equal(raw, raw2)
    # the weight gradient, from hidden layers as the forward wrote them
    g = rng.normal(size=(n, 4)).astype(np.float32)
    h = _np(hid)
    h[m:] = 0
    grad = torch.full((len(counts), E.N_CELL), 7.0, device="cuda")
    work = torch.empty(nb.nerf_cells_backward_workspace(n, len(counts)), device="cuda", dtype=torch.uint8)
    hid[m:] = float("nan")                               # not looked at
    gt = _cuda(torch, g)
    gt[m:] = float("nan")
    nb.nerf_cells_backward(xt, dt, ot, wt, hid, gt, grad, work)
    ref = E.cells_backward(x, d, offset, w, h, g)
    bound = np.zeros_like(ref)
    for c in range(len(counts)):
        r = slice(offset[c], offset[c + 1])
        _, _, w2, _, ws, _, wc, _ = E.cell_parts(w[c])
        gc, gs = np.abs(g[r, :3].astype(np.float64)), np.abs(g[r, 3].astype(np.float64))
        on1, on2 = h[r, :32] > 0, h[r, 32:] > 0
        m2 = (gc @ np.abs(wc[:, :32]) + gs[:, None] * np.abs(ws)) * on2
        e2 = (C3 + 5 * U) * m2
        m1 = ((m2 + e2) @ np.abs(w2)) * on1
        e1 = (e2 @ np.abs(w2)) * on1 + (C3 + 34 * U) * m1
        acc = C3 + (counts[c] + 8) * U                   # a sum over the cell's rows, in any order
        apx, both = np.abs(px[r]), np.concatenate([h[r, 32:], np.abs(pd[r])], axis=1)
        eb = np.concatenate([np.zeros((counts[c], 32)), ed[r]], axis=1)
        M1, M2 = m1 + e1, m2 + e2
        one = np.ones((counts[c], 1))

        def outer(a, ea, b, eb_):
            return a.T @ eb_ + ea.T @ (b + eb_) + acc * (a.T @ (b + eb_))

        z32, z1, z4 = np.zeros((counts[c], 32)), np.zeros((counts[c], 1)), np.zeros((counts[c], 3))
        bound[c] = np.concatenate([
            outer(M1, e1, apx, ex[r]).ravel(), outer(M1, e1, one, z1).ravel(), outer(M2, e2, h[r, :32], z32).ravel(),
            outer(M2, e2, one, z1).ravel(), outer(gs[:, None], z1, h[r, 32:], z32).ravel(), outer(gs[:, None], z1, one, z1).ravel(),
            outer(gc, z4, both, eb).ravel(), outer(gc, z4, one, z1).ravel()])
    _near(_np(grad), ref, 1.01 * bound + 1e-30, "grad")
    again = torch.full_like(grad, -3.0)
    nb.nerf_cells_backward(xt, dt, ot, wt, hid, gt, again, work)
    assert torch.equal(grad, again)


def test_a_rows_value_does_not_depend_on_its_neighbours(torch):
    """The same rows in one cell, and cut into cells of one to 70 rows that have the same weights: the same bits."""
    import neural_radiance_field_b200 as nb
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    counts = [1, 2, 7, 8, 9, 0, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 70, 127, 128, 129, 160, 161]
    n = sum(counts)
    x, d, w = rnd(n, 3), rnd(n, 3), rnd(1, 3317) * 0.1
    outs = []
    for off in ([0, n], np.concatenate([[0], np.cumsum(counts)])):
        off = _cuda(torch, np.asarray(off, dtype=np.int32))
        raw, hidden = torch.full((n, 4), 7.0, device="cuda"), torch.full((n, 64), 7.0, device="cuda")
        nb.nerf_cells_forward(x, d, off, w.expand(off.numel() - 1, -1).contiguous(), raw, hidden)
        outs.append((raw, hidden))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("cells", [1, 3, 64, 200, 591])
def test_cell_gradients_of_few_cells(torch, cells):
    """Few cells have their parts summed in slices: the bits that they get among 1,000 cells of which the rest is
    empty, and biases that are the plain sums of d_raw. Of the magnitudes' sum: 4 U for a value as two tf32 numbers
    (the lower one's own rounding, 2^-11 of 2^-11), 6 x 16 U for a tile's six matrix instructions (eight truncated
    terms each, 2 U a term), then at most one rounded addition a row."""
    import neural_radiance_field_b200 as nb
    gen = torch.Generator(device="cuda").manual_seed(cells)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    n = 30000
    x, d, w, d_raw = rnd(n, 3), rnd(n, 3), rnd(1000, 3317) * 0.1, rnd(n, 4)
    off = np.concatenate([[0], np.sort(np.random.default_rng(cells).integers(0, n + 1, cells - 1)), [n]])
    grads = []
    for many in (cells, 1000):
        o = _cuda(torch, np.concatenate([off, np.full(many - cells, n)]).astype(np.int32))
        raw, hidden = torch.empty(n, 4, device="cuda"), torch.empty(n, 64, device="cuda")
        nb.nerf_cells_forward(x, d, o, w[:many], raw, hidden)
        grads.append(torch.full((many, 3317), float("nan"), device="cuda"))
        work = torch.empty(nb.nerf_cells_backward_workspace(n, many), device="cuda", dtype=torch.uint8)
        nb.nerf_cells_backward(x, d, o, w[:many], hidden, d_raw, grads[-1], work)
    assert torch.equal(grads[0], grads[1][:cells]) and grads[1][cells:].eq(0).all()
    got, terms = _np(grads[0]), _np(d_raw)
    for c in range(cells):
        rows = terms[off[c]:off[c + 1]]
        bound = (len(rows) + 100) * U * np.abs(rows).sum(0)
        _near(got[c, 3314:3317], rows[:, :3].sum(0), bound[:3], "color biases")
        _near(got[c, 3136:3137], rows[:, 3:].sum(0), bound[3:], "sigma bias")


def test_cell_gradients_back_to_back_share_a_workspace(torch):
    """Launch follows launch with other rows per cell and one workspace: every result is that of the call alone."""
    import neural_radiance_field_b200 as nb
    cases, n = [], 4000
    for seed, counts in enumerate(([4000], [7, 0, 1993, 2000], [100] * 40)):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
        counts = counts + [0] * (41 - len(counts))
        off = _cuda(torch, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        x, d, w, d_raw = rnd(n, 3), rnd(n, 3), rnd(41, 3317) * 0.1, rnd(n, 4)
        raw, hidden = torch.empty(n, 4, device="cuda"), torch.empty(n, 64, device="cuda")
        nb.nerf_cells_forward(x, d, off, w, raw, hidden)
        cases.append((x, d, off, w, hidden, d_raw))
    size = nb.nerf_cells_backward_workspace(n, 41)
    alone = []
    for c in cases:
        g = torch.full((41, 3317), float("nan"), device="cuda")
        nb.nerf_cells_backward(*c, g, torch.zeros(size, device="cuda", dtype=torch.uint8))
        torch.cuda.synchronize()
        assert torch.isfinite(g).all()
        alone.append(g)
    work = torch.empty(size, device="cuda", dtype=torch.uint8)
    outs = [torch.full((41, 3317), float("nan"), device="cuda") for _ in range(30)]
    for r, g in enumerate(outs):
        nb.nerf_cells_backward(*cases[r % 3], g, work)
    for r, g in enumerate(outs):
        assert torch.equal(g, alone[r % 3])


def test_cells_far_positions(torch):
    """Positions far outside the grid: the angles' quadrants are still exact."""
    import neural_radiance_field_b200 as nb
    x = np.array([[100.25, -2999.7, 0.1], [2.0 ** 23, 3.0, -2.0 ** 24], [-1023.5, 511.75, 4095.0625], [0.0, -0.0, 1e-30]], np.float32)
    d = np.array([[1, 2, 3], [0, 0, -2], [1e-20, 1e-20, 0], [1e18, 0, 1e18]], np.float32)
    w = kilonerf_weights(3, n_cells=1)
    off = np.array([0, 4], np.int32)
    raw, hid = torch.empty(4, 4, device="cuda"), torch.empty(4, 64, device="cuda")
    nb.nerf_cells_forward(_cuda(torch, x), _cuda(torch, d), _cuda(torch, off), _cuda(torch, w), raw, hid)
    r_raw, r_hid = E.cells_forward(x, d, off, w)
    # the layers' bound of test_cells, over the largest input of a row; and the oracle's own angle, pi v in fp64:
    # 2^-53 * pi * 512 * 2^24 = 3e-6 at most
    e = 64 * (4.5 * 2.0 ** -23 + 3e-6) + (C3 + 66 * U) * (60 + np.abs(x).sum(1, keepdims=True))
    assert (np.abs(_np(hid) - r_hid) <= 33 * e).all()


def _cells_once(torch, x, d, off, w):
    import neural_radiance_field_b200 as nb
    raw, hid = torch.full((len(x), 4), 7.0, device="cuda"), torch.full((len(x), 64), 7.0, device="cuda")
    nb.nerf_cells_forward(_cuda(torch, x), _cuda(torch, d), _cuda(torch, off), _cuda(torch, w), raw, hid)
    return raw, hid


@pytest.mark.parametrize("rows", [5, 40, 200])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_cells_that_are_not_finite_show_it(torch, rows, bad):
    """NaN or infinity in one row's position: NaN in that row's hidden layers and outputs; in its direction: in its
    colours; in one weight of one cell: in what that cell computes from it. Every other row keeps its bits."""
    rng, off, x, d, w = _cells_case(torch, rows, [rows, rows + 3, 0, rows])
    raw, hid = _cells_once(torch, x, d, off, w)
    assert torch.isfinite(raw).all() and torch.isfinite(hid).all()
    same = lambda a, b, r: torch.equal(a[r], b[r])  # noqa: E731
    for r in (0, rows - 1, rows + 2, 2 * rows + 3):
        others = torch.arange(len(x), device="cuda") != r
        for c in range(3):
            x2 = x.copy()
            x2[r, c] = bad
            raw2, hid2 = _cells_once(torch, x2, d, off, w)
            assert torch.isnan(hid2[r]).all() and torch.isnan(raw2[r]).all()
            assert same(raw, raw2, others) and same(hid, hid2, others)
            d2 = d.copy()
            d2[r, c] = bad
            raw2, hid2 = _cells_once(torch, x, d2, off, w)
            assert torch.isnan(raw2[r, :3]).all() and raw2[r, 3] == raw[r, 3] and torch.equal(hid, hid2) and same(raw, raw2, others)
    mine = torch.zeros(len(x), device="cuda", dtype=torch.bool)
    mine[rows:2 * rows + 3] = True
    f = 9                                                # the feature whose weight is not finite
    b1 = 32 * 63 + f
    b2 = 32 * 63 + 32 + 32 * 32 + f
    for at, layer in ((f * 63 + 20, 1), (b1, 1), (32 * 63 + 32 + f * 32 + 3, 2), (b2, 2)):   # W1, b1, W2, b2
        w2 = w.copy()
        w2[1, at] = bad
        raw2, hid2 = _cells_once(torch, x, d, off, w2)
        assert same(raw, raw2, ~mine) and same(hid, hid2, ~mine)
        if at in (b1, b2) and bad == -np.inf:    # a bias of -inf turns its feature off
            off1 = hid2[mine, 32 * (layer - 1) + f]
            assert off1.eq(0).all()
            continue
        hit = hid2[mine]
        assert (~torch.isfinite(hit[:, 32 * (layer - 1) + f])).all() and (~torch.isfinite(raw2[mine])).all()
        if layer == 2:
            assert same(hid[:, :32], hid2[:, :32], mine)


@pytest.mark.parametrize("rows", [5, 200])
def test_cell_gradients_that_are_not_finite_show_it(torch, rows):
    """A row with a NaN position: NaN in the gradients of its cell's weights on gamma(x) and on the hidden layers; the
    bits of every other cell's gradient stay."""
    import neural_radiance_field_b200 as nb
    rng, off, x, d, w = _cells_case(torch, rows, [rows, rows + 3, 0, rows])
    g = _cuda(torch, rng.normal(size=(len(x), 4)).astype(np.float32))
    work = torch.empty(nb.nerf_cells_backward_workspace(len(x), 4), device="cuda", dtype=torch.uint8)
    grads = []
    for bad in (False, True):
        if bad:
            x[rows + 1, 2] = np.nan
        _, hid = _cells_once(torch, x, d, off, w)
        grads.append(torch.full((4, E.N_CELL), 7.0, device="cuda"))
        nb.nerf_cells_backward(_cuda(torch, x), _cuda(torch, d), _cuda(torch, off), _cuda(torch, w), hid, g, grads[-1], work)
    assert torch.isfinite(grads[0]).all()
    assert all(torch.equal(grads[0][c], grads[1][c]) for c in (0, 2, 3))
    w1, _, w2, _, ws, _, wc, _ = torch.split(grads[1][1], [2016, 32, 1024, 32, 32, 1, 177, 3])
    z = w1.view(32, 63)                                  # coordinate 2 and its angles; the others' factors stay finite
    cols = [2, *range(23, 33), *range(53, 63)]
    assert torch.isnan(z[:, cols]).all()
    assert torch.isnan(w2).all() and torch.isnan(ws).all() and torch.isnan(wc.view(3, 59)[:, :32]).all()


def test_cells_directions_of_every_length(torch):
    """Directions from the smallest floats to the largest: the colours are the unit direction's, whose coordinates are
    within 3.5u each, through gamma(d) and the head (the bounds of test_cells; the layers below are the same)."""
    length = np.array([2.0 ** e for e in (-148, -140, -130, -126, -100, -75, -64, -63, -40, 0, 40, 62, 63, 64, 90, 120, 126)])
    base = np.random.default_rng(4).normal(size=(len(length), 3))
    base /= np.abs(base).max(1, keepdims=True)
    d = (base * length[:, None]).astype(np.float32)
    d = np.concatenate([d, np.float32([[3.4e38, -3.4e38, 3.4e38], [0, 0, 1e-45], [0, -2.0 ** 127, 0], [1e-20, 1e-20, 0], [1e18, 0, 1e18],
                                       [1e30, 1e-30, 1e10], [-1e-42, 1e-44, 1.0]])])
    n = len(d)
    x = np.tile(np.float32([[0.3, -0.2, 0.9]]), (n, 1))
    w, off = kilonerf_weights(9, n_cells=1), np.array([0, n], np.int32)
    raw, hid = _cells_once(torch, x, d, off, w)
    assert (hid == hid[0]).all() and (raw[:, 3] == raw[0, 3]).all()
    _, _, _, _, _, _, wc, bc = (np.abs(v) for v in E.cell_parts(w[0]))
    _, pd = E.encodings(x, d)
    _, ed = _encoding_errors(x, d.astype(np.float64))
    h2 = _np(hid)[:, 32:]                                # the head's other inputs, as the call wrote them
    _, _, _, _, _, _, swc, sbc = E.cell_parts(w[0])
    ref = np.concatenate([h2, pd], axis=1) @ swc.T + sbc
    mag = np.concatenate([h2, np.abs(pd) + ed], axis=1) @ wc.T + bc
    _near(_np(raw)[:, :3], ref, 1.01 * (ed @ wc[:, 32:].T + 62 * U * mag), "colours")
    # and in the weight gradient, of which a row alone in its cell with d_raw = (1, 0, 0, 0) shows gamma(d): a product
    # with 1 of two tf32 parts (the lower one cut, 2^-21), two truncated sums with zeros (2U each), one rounded. Of a
    # coordinate below the normal range (one is 1e-60, which is 0 in fp32) the parts' steps are 2^-136 or the parts 0:
    # 2^-126
    import neural_radiance_field_b200 as nb
    d_raw = torch.zeros(n, 4, device="cuda")
    d_raw[:, 0] = 1
    grad = torch.full((n, E.N_CELL), 7.0, device="cuda")
    work = torch.empty(nb.nerf_cells_backward_workspace(n, n), device="cuda", dtype=torch.uint8)
    nb.nerf_cells_backward(_cuda(torch, x), _cuda(torch, d), torch.arange(n + 1, device="cuda", dtype=torch.int32),
                           _cuda(torch, np.repeat(w, n, axis=0)), hid, d_raw, grad, work)
    _near(_np(grad)[:, 3137 + 32:3137 + 59], pd, 1.01 * (ed + (2.0 ** -21 + 5 * U) * (np.abs(pd) + ed)) + 2.0 ** -126, "gradient of the head")


def test_cells_encodings_of_far_positions(torch):
    """Each column of gamma(x), read out by cells whose first layer is one of its columns and its negative, with the
    sines of angles that are exact: k pi v with 2^k v taken modulo 2 before anything is rounded. The product with 1
    reads the value as its two tf32 parts, the lower one cut at 2^-10 of its 2^-11; its sum with zeros truncates
    twice, 2U each."""
    x = np.float32([[0.3, -1.4999, 0.7], [100.25, -2999.7, 0.1], [2.0 ** 23, 3.0, -2.0 ** 24], [-1023.5, 511.75, 4095.0625],
                    [0.0, -0.0, 1e-30], [8388607.5, -8388608.0, 16777215.0], [65535.996, -32767.502, 1048575.94],
                    [2.0 ** 30, -2.0 ** 60, 2.0 ** 100], [12345.678, -0.5, 33554434.0]])
    n, cells = len(x), 4
    w = np.zeros((cells, E.N_CELL), np.float32)
    for c in range(cells):
        w1 = w[c, :2016].reshape(32, 63)
        for j in range(16):
            if 16 * c + j < 63:
                w1[j, 16 * c + j], w1[16 + j, 16 * c + j] = 1.0, -1.0
    d = np.tile(np.float32([[0, 0, 1]]), (n * cells, 1))
    off = (n * np.arange(cells + 1)).astype(np.int32)
    # far columns of x itself are left out of their rows' sums only by a weight of 0; they are finite
    _, hid = _cells_once(torch, np.tile(x, (cells, 1)), d, off, w)
    h = _np(hid)[:, :32].reshape(cells, n, 2, 16)
    assert ((h[:, :, 0] == 0) | (h[:, :, 1] == 0)).all()
    got = (h[:, :, 0] - h[:, :, 1]).transpose(1, 0, 2).reshape(n, 64)[:, :63]
    half = np.fmod(x.astype(np.float64)[:, :, None] * 2.0 ** np.arange(10), 2.0).reshape(n, 30)
    ref = np.concatenate([x, np.sin(np.pi * half), np.cos(np.pi * half)], axis=1)
    ex = _encoding_errors(x, np.ones((n, 3)))[0]
    _near(got, ref, 1.01 * (ex + (2.0 ** -21 + 4 * U) * np.abs(ref)) + 4e-16, "gamma(x)")


def test_cells_agree_with_the_renderers_network(torch):
    """sigma and rgb of one KiloNeRF frame: each ray marched by hand through nerf_test_march's live samples,
    nerf_expert_sort and nerf_cells_forward composites to nerf_render's colour."""
    import dataclasses
    import nerf_inputs as S
    import neural_radiance_field_b200 as nb
    from oracle import nerf as onerf
    wl = dataclasses.replace(S.WORKLOADS["kilonerf"], H=6, W=8, focal=10.0, ert_T=0.0)
    packed, _ = S.occupancy_grid(7)
    w = kilonerf_weights(8)
    o, d = onerf.raygen(wl.H, wl.W, wl.focal, wl.c2w())
    o, d = _cuda(torch, o), _cuda(torch, d)
    occ, wt, R = _cuda(torch, packed.view(np.int32)).view(torch.uint32), _cuda(torch, w), wl.n_rays
    with nb.Renderer(model=nb.NERF_MODEL_KILONERF, max_rays=R, max_samples=wl.n_coarse) as rnd:
        p = rnd.params(occupancy=occ, cell_w=wt, march_step=wl.march_step, ert_T=0.0)
        rgb, dep, acc = torch.empty(R, 3, device="cuda"), torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
        rnd.render(o, d, wl.near, wl.far, wl.n_coarse, 0, p, rgb, dep, acc)
        rnd.sync_status()
    cnt, live = torch.empty(R, device="cuda", dtype=torch.int32), torch.empty(R, wl.n_coarse, device="cuda", dtype=torch.uint8)
    nb.nerf_test_march(o, d, wl.near, wl.march_step, wl.n_coarse, occ, cnt, live)
    ray, k = live.nonzero(as_tuple=True)
    t = torch.tensor(wl.near, device="cuda") + k.float() * torch.tensor(wl.march_step, device="cuda")
    x = o[ray] + t[:, None] * d[ray]
    n = x.shape[0]
    assert n > 300
    cell = torch.empty(n, device="cuda", dtype=torch.int32)
    i32 = torch.int32
    nb.nerf_test_route_cells(x.contiguous(), cell, torch.empty(4096, device="cuda", dtype=i32), torch.empty(4097, device="cuda", dtype=i32))
    off, _, pos = _sorted(torch, cell[:, None].contiguous(), 4096)
    xs, ds, raws, raw = (torch.empty(n, c, device="cuda") for c in (3, 3, 4, 4))
    nb.nerf_expert_dispatch(x.contiguous(), pos, xs)
    nb.nerf_expert_dispatch(d[ray].contiguous(), pos, ds)
    nb.nerf_cells_forward(xs, ds, off, wt, raws)
    nb.nerf_expert_combine(raws, pos, raw)
    a = raw.double()
    delta = wl.march_step * d.double().norm(dim=1)[ray]
    tau = a[:, 3].clamp_min(0) * delta
    total = torch.zeros(R, device="cuda", dtype=torch.float64)
    want = torch.zeros(R, 3, device="cuda", dtype=torch.float64)
    start = 0
    for r, c in enumerate(cnt.tolist()):
        s = slice(start, start + c)
        T = torch.exp(-(tau[s].cumsum(0) - tau[s]))
        want[r] = ((T * -torch.expm1(-tau[s]))[:, None] * torch.sigmoid(a[s, :3])).sum(0)
        start += c
    # the parity bar of the fp32 render; both sides are within it of the same field
    assert (rgb.double() - want).abs().max() <= 1e-4


# ------------------------------------------------------------------ together

def _mixture(torch, seed, n=400, k=3, e=6):
    """A mixture over e cell networks: gate logits -> top k -> sort -> networks -> weighted blend."""
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(n, e))
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    ids[rng.random((n, k)) < 0.1] = -1
    ids[5] = -1
    w = rng.random((n, k)).astype(np.float32)
    x, d = rng.uniform(-1.5, 1.5, size=(n, 3)).astype(np.float32), rng.normal(size=(n, 3)).astype(np.float32)
    return rng, ids, w, x, d, kilonerf_weights(seed, n_cells=e)


class _Step:
    """One training step of the mixture with its buffers; run() only enqueues."""

    def __init__(self, torch, ids, w, x, d, cells, G):
        import neural_radiance_field_b200 as nb
        n, k = ids.shape
        e, m = len(cells), n * k
        self.torch, self.nb, self.e = torch, nb, e
        self.ids, self.w, self.x, self.d, self.cells, self.G = (_cuda(torch, a) for a in (ids, w, x, d, cells, G))
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        i32 = torch.int32
        self.off, self.pos = z(e + 1).to(i32), z(n, k).to(i32)
        self.xs, self.ds, self.raws, self.hid, self.out = z(m, 3), z(m, 3), z(m, 4), z(m, 64), z(n, 4)
        self.d_raws, self.dw, self.grad = z(m, 4), z(n, k), z(e, E.N_CELL)
        self.sw = torch.empty(nb.nerf_expert_sort_workspace(n, k, e), device="cuda", dtype=torch.uint8)
        self.cw = torch.empty(nb.nerf_cells_backward_workspace(m, e), device="cuda", dtype=torch.uint8)

    def run(self, stream=None):
        nb, a = self.nb, dict(stream=stream)
        nb.nerf_expert_sort(self.ids, self.e, self.off, None, self.pos, self.sw, **a)
        nb.nerf_expert_dispatch(self.x, self.pos, self.xs, **a)
        nb.nerf_expert_dispatch(self.d, self.pos, self.ds, **a)
        nb.nerf_cells_forward(self.xs, self.ds, self.off, self.cells, self.raws, self.hid, **a)
        nb.nerf_expert_combine(self.raws, self.pos, self.out, self.w, **a)
        nb.nerf_expert_combine_backward(self.G, self.raws, self.pos, self.d_raws, self.w, self.dw, **a)
        nb.nerf_cells_backward(self.xs, self.ds, self.off, self.cells, self.hid, self.d_raws, self.grad, self.cw, **a)

    def results(self):
        return [t.clone() for t in (self.out, self.dw, self.grad)]


def test_a_training_step_of_a_mixture(torch):
    """The whole chain against the oracle's chain and against differences of its loss."""
    rng, ids, w, x, d, cells = _mixture(torch, 3)
    n, k = ids.shape
    G = rng.normal(size=(n, 4)).astype(np.float32)
    step = _Step(torch, ids, w, x, d, cells, G)
    step.run()
    out, dw, grad = (_np(t) for t in step.results())
    off, order, pos = E.sort(ids, len(cells))
    zero = np.zeros((n * k, 3))

    def chain(w, cells):
        xs, ds = E.dispatch(x, pos, None, zero), E.dispatch(d, pos, None, np.ones((n * k, 3)))
        raws, hid = E.cells_forward(xs, ds, off, cells)
        return E.combine(raws, pos, w), raws, hid, xs, ds

    r_out, raws, hid, xs, ds = chain(w.astype(np.float64), cells.astype(np.float64))
    # measured values of O(1) through three fp32 layers: 1e-4 of the largest, the bar of the fp32 parity tests
    assert np.abs(out - r_out).max() <= 1e-4 * np.abs(r_out).max() and (out[5] == 0).all()
    r_dw = E.dots(raws, G, pos)
    assert np.abs(dw - r_dw).max() <= 1e-4 * np.abs(r_dw).max()
    d_raws = E.dispatch(G, pos, w, np.zeros((n * k, 4)))
    r_grad = E.cells_backward(xs, ds, off, cells, hid, d_raws)
    assert np.abs(grad - r_grad).max() <= 1e-4 * np.abs(r_grad).max()
    for q in rng.integers(0, E.N_CELL, size=6).tolist() + [3314]:
        hi, lo = cells.astype(np.float64), cells.astype(np.float64)
        hi[1, q] += 1e-6
        lo[1, q] -= 1e-6
        num = ((chain(w, hi)[0] - chain(w, lo)[0]) * G).sum() / 2e-6
        assert abs(num - grad[1, q]) <= 1e-4 * np.abs(r_grad).max() + 1e-5


def test_two_steps_on_two_streams_and_a_captured_one(torch):
    """Steps that overlap on two streams, and a step replayed from a CUDA graph on new inputs while another
    runs, give what each gives alone."""
    steps, want = [], []
    for seed in (11, 12):
        rng, ids, w, x, d, cells = _mixture(torch, seed, n=3000)
        G = rng.normal(size=(3000, 4)).astype(np.float32)
        steps.append(_Step(torch, ids, w, x, d, cells, G))
        steps[-1].run()
        want.append(steps[-1].results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in steps:
        s.out.zero_(), s.grad.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        steps[0].run()
    for t in ("ids", "w", "x", "d", "cells", "G"):       # the graph reads these buffers: the other step's inputs
        getattr(steps[0], t).copy_(getattr(steps[1], t))
    steps[0].out.zero_(), steps[0].grad.zero_()
    torch.cuda.synchronize()
    g.replay()
    steps[1].run(stream=streams[1])
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(steps[0].results(), want[1]))
    assert all(torch.equal(a, b) for a, b in zip(steps[1].results(), want[1]))


def test_every_operator_in_a_graph(torch):
    """Each call captured on a side stream, with its inputs changed before the replay: what an eager call on
    those inputs gives; at sizes of the one-launch and the many-launch forms, clusters among them."""
    import neural_radiance_field_b200 as nb
    f32, i32 = torch.float32, torch.int32
    g = torch.Generator(device="cuda")
    g.manual_seed(4)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    def check(ins, outs, call):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        call()
        with torch.cuda.graph(graph, stream=st):
            call()
        for t in ins:
            t.copy_(t.flip(0).clone())
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(-3)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))

    for n, k, e in ((20, 8, 300), (40000, 2, 4096)):
        ids = torch.randint(0, e, (n, k), generator=g, device="cuda", dtype=i32)
        off, order, pos = torch.empty(e + 1, device="cuda", dtype=i32), torch.empty(n * k, device="cuda", dtype=i32), torch.empty(n, k, device="cuda", dtype=i32)
        work = torch.empty(nb.nerf_expert_sort_workspace(n, k, e), device="cuda", dtype=torch.uint8)
        check([ids], [off, order, pos], (lambda: nb.nerf_expert_sort(ids, e, off, order, pos, work)))
        x, rows, w, out, dw = rnd(n, 36), rnd(n * k, 36), rnd(n, k), rnd(n, 36), rnd(n, k)
        check([x, w], [rows], (lambda: nb.nerf_expert_dispatch(x, pos, rows, w)))
        check([rows, w], [out], (lambda: nb.nerf_expert_combine(rows, pos, out, w)))
        check([rows, x], [out, dw], (lambda: nb.nerf_expert_dispatch_backward(rows, x, pos, out, w, dw)))
        dr = rnd(n * k, 36)
        check([rows, x], [dr, dw], (lambda: nb.nerf_expert_combine_backward(x, rows, pos, dr, w, dw)))
    for n, e, dt in ((30, 100, f32), (2000, 4096, torch.bfloat16), (400, 40000, f32), (9, 130000, torch.float16), (3, 300000, f32)):
        s, tl = rnd(n, e).to(dt), rnd(n, 5)
        ti = torch.randint(0, e, (n, 5), generator=g, device="cuda", dtype=i32)
        loss, grad = torch.empty(n, device="cuda"), torch.empty(n, e, device="cuda", dtype=dt)
        check([s, tl, ti], [loss, grad], (lambda: nb.nerf_distill_topk(s, tl, ti, 1.3, loss, grad)))
    n, e = 3000, 20
    x, d, dr, w = rnd(n, 3), rnd(n, 3), rnd(n, 4), rnd(e, 3317) / 6
    off = torch.linspace(0, n, e + 1, device="cuda").int()
    raw, hid, grad = rnd(n, 4), rnd(n, 64), torch.empty(e, 3317, device="cuda")
    work = torch.empty(nb.nerf_cells_backward_workspace(n, e), device="cuda", dtype=torch.uint8)
    check([x, d, w], [raw, hid], (lambda: nb.nerf_cells_forward(x, d, off, w, raw, hid)))
    check([x, d, dr], [grad], (lambda: nb.nerf_cells_backward(x, d, off, w, hid, dr, grad, work)))


def test_a_gate_learns_from_its_teachers_top_logits(torch):
    """The gate's logits step along the distillation gradient; what the kernel returns is the gradient of the
    summed loss along that direction, by differences of the oracle's loss."""
    import neural_radiance_field_b200 as nb
    rng = np.random.default_rng(21)
    n, e, k = 200, 512, 8
    s, teacher = rng.normal(size=(n, e)).astype(np.float32), (2 * rng.normal(size=(n, k))).astype(np.float32)
    ids = np.stack([rng.permutation(e)[:k] for _ in range(n)]).astype(np.int32)
    loss, grad = torch.empty(n, device="cuda"), torch.empty(n, e, device="cuda")
    nb.nerf_distill_topk(_cuda(torch, s), _cuda(torch, teacher), _cuda(torch, ids), 2.0, loss, grad)
    g = _np(grad)
    f = lambda a: E.distill(s.astype(np.float64) + a * g, teacher.astype(np.float64), ids, 2.0)[0].sum()  # noqa: E731
    # central difference of a smooth function: error h^2 |f'''| / 6 with h = 1e-3 and |f'''| <= 8 sum|g|^3 / T
    num, dot = (f(1e-3) - f(-1e-3)) / 2e-3, (g * g).sum()
    assert abs(num - dot) <= 1e-6 * 8 * (np.abs(g).sum(1) ** 3).sum() + 1e-5 * dot


def test_offsets_past_32_bits(torch):
    """Rows whose byte and element offsets pass 2^32."""
    import neural_radiance_field_b200 as nb
    n, width = 4200, 1 << 20
    x = torch.zeros(n, width, device="cuda", dtype=torch.bfloat16)             # 4.4e9 elements, 8.8 GB
    x[-1] = 3.0
    x[0, -1] = 5.0
    pos = torch.arange(n - 1, -1, -1, device="cuda", dtype=torch.int32)[:, None].contiguous()
    rows = torch.zeros_like(x)
    nb.nerf_expert_dispatch(x, pos, rows)
    assert rows[0].eq(3).all() and rows[-1, -1] == 5 and rows[-1, :-1].eq(0).all() and rows[n // 2].eq(0).all()
    x.zero_()
    nb.nerf_expert_combine(rows, pos, x)
    assert x[-1].eq(3).all() and x[0, -1] == 5 and x[0, :-1].eq(0).all()
    loss = torch.empty(n, device="cuda")
    tl, ti = torch.zeros(n, 1, device="cuda"), torch.full((n, 1), width - 1, device="cuda", dtype=torch.int32)
    nb.nerf_distill_topk(x, tl, ti, 1.0, loss, rows)
    # row 0: q of the class is e^5 / (2^20 - 1 + e^5) = 1.4e-4, and -(1 - 1.4e-4) is nearest to -1 among bf16
    # values (the next is -1 + 2^-8); the other classes have q = 1 / (2^20 - 1 + e^5), in row 0 and (3s alone) 2^-20
    assert rows[-1, -1] == -1 and rows[0, -1] == -1 and torch.isfinite(loss).all()
    assert abs(rows[0, 0].item() * (width - 1 + np.exp(5)) - 1) <= 2.0 ** -8 and rows[-1, :-1].eq(2.0 ** -20).all()
