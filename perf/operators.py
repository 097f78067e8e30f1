"""Measured cases of the expert operators: the sort of (point, expert) pairs by
expert, rows taken to that order and back with their weights and gradients, the
distillation loss against a teacher's top logits, and the per-cell networks on
sorted rows with their weight gradient.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and the calls of neural_radiance_field_b200.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CELLS = 4096          # the 16^3 cells of the per-cell networks
CELL_PARAMS = 3317    # W1[32][63] b1[32] W2[32][32] b2[32] ws[32] bs[1] Wc[3][59] bc[3]


def listed():
    return [
        # One point blended from the eight cells around it: a single-token call.
        {"name": "sort_point", "op": "sort", "n": 1, "k": 8, "experts": CELLS, "routing": "cells"},
        # A training batch: 4096 rays of 192 samples, each in the eight cells around it.
        {"name": "sort_batch", "op": "sort", "n": 786432, "k": 8, "experts": CELLS, "routing": "cells"},
        # 256-wide features of a batch's coarse samples to their two experts of 64.
        {"name": "dispatch_batch", "op": "dispatch", "n": 262144, "k": 2, "experts": 64, "width": 256,
         "dtype": "bf16", "weighted": False, "routing": "gate"},
        # The 63-wide encoded positions of one ray and a sample: gradients of a weighted dispatch.
        {"name": "dispatch_ray_backward", "op": "dispatch_backward", "n": 193, "k": 2, "experts": 64, "width": 63,
         "dtype": "fp32", "weighted": True, "routing": "gate"},
        # (r, g, b, sigma) of eight cells blended per sample of a training batch.
        {"name": "combine_raw", "op": "combine", "n": 786432, "k": 8, "experts": CELLS, "width": 4,
         "dtype": "fp32", "weighted": True, "routing": "cells"},
        # Gradients of a weighted combination of 256-wide expert outputs.
        {"name": "combine_batch_backward", "op": "combine_backward", "n": 262144, "k": 2, "experts": 64, "width": 256,
         "dtype": "bf16", "weighted": True, "routing": "gate"},
        # One point's gate logits over all cells against a teacher's top eight: loss alone.
        {"name": "distill_point", "op": "distill", "n": 1, "k": 8, "experts": CELLS, "dtype": "fp32", "grad": False},
        # A batch of gate logits over all cells, loss and gradient.
        {"name": "distill_batch", "op": "distill", "n": 65536, "k": 16, "experts": CELLS, "dtype": "bf16", "grad": True},
        # Few rows of many classes, an odd number of them.
        {"name": "distill_wide", "op": "distill", "n": 777, "k": 32, "experts": 100003, "dtype": "fp32", "grad": True},
        # The per-cell networks on one ray's samples, as a render calls them.
        {"name": "cells_ray", "op": "cells", "n": 192, "experts": CELLS, "routing": "ray", "store": False},
        # The per-cell networks on a training batch, each sample in its own cell, with the hidden
        # layers kept for the backward pass; and the weight gradient from them.
        {"name": "cells_batch", "op": "cells", "n": 786432, "experts": CELLS, "routing": "cells", "store": True},
        {"name": "cells_batch_backward", "op": "cells_backward", "n": 786432, "experts": CELLS, "routing": "cells"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch_backward", "combine", "combine_backward", "distill", "distill", "cells",
                     "cells_backward"])
    if op == "sort":
        cells = rng.random() < 0.4
        k = 8 if cells else rng.choice([1, 2, 3, 4, 6, 8])
        return {"op": op, "n": _log(rng, 1, 786432), "k": k, "experts": CELLS if cells else _log(rng, 8, CELLS),
                "routing": "cells" if cells else "gate"}
    if op == "distill":
        e = _log(rng, 8, 100003)
        return {"op": op, "n": _log(rng, 1, max(2, min(65536, 77000000 // e))), "k": rng.randint(1, min(32, e)),
                "experts": e, "dtype": rng.choice(["fp32", "bf16", "fp16"]), "grad": rng.random() < 0.7}
    if op in ("cells", "cells_backward"):
        e = rng.choice([CELLS, CELLS, _log(rng, 8, 2000)])
        case = {"op": op, "n": _log(rng, 1, 786432), "experts": e, "routing": "cells" if e == CELLS else "gate"}
        return {**case, "store": rng.random() < 0.5} if op == "cells" else case
    width = rng.choice([3, 4, 27, 32, 63, 64, 90, 128, 256, _log(rng, 1, 1024)])
    k = rng.choice([1, 2, 3, 4, 8])
    cells = k == 8 and rng.random() < 0.5
    return {"op": op, "n": _log(rng, 1, max(2, min(786432, 134000000 // (width * k)))), "k": k,
            "experts": CELLS if cells else _log(rng, 8, 512), "width": width,
            "dtype": rng.choice(["fp32", "bf16", "fp16"]), "weighted": rng.random() < 0.7,
            "routing": "cells" if cells else "gate"}


# ----------------------------------------------------------------- inputs

def _ball(n, g):
    """n points in the ball of radius 1.5."""
    v = torch.randn(n, 3, generator=g, device="cuda")
    r = 1.4999 * torch.rand(n, 1, generator=g, device="cuda") ** (1.0 / 3.0)
    return v * (r / v.norm(dim=1, keepdim=True).clamp_min(1e-20))


def _segments(n, g):
    """n points as runs of 64 samples along segments that cross the ball: neighbours share cells."""
    rays = -(-n // 64)
    a, b = _ball(rays, g), _ball(rays, g)
    t = (torch.arange(64, device="cuda") + 0.5) / 64
    return (a[:, None] + (b - a)[:, None] * t[None, :, None]).reshape(-1, 3)[:n].contiguous()


def _route(case, g):
    """ids [n][k] int32 (-1: dropped) and weights [n][k] of each point's experts."""
    n, k, e = case["n"], case["k"], case["experts"]
    if case["routing"] == "cells":   # the eight cells around a point, trilinear weights; none beyond the grid
        u = (_segments(n, g) + 1.5) * (16.0 / 3.0) - 0.5
        lo = u.floor()
        f = u - lo
        bits = torch.tensor([[i >> 2 & 1, i >> 1 & 1, i & 1] for i in range(8)], device="cuda")
        c = lo[:, None].long() + bits[None]
        w = torch.where(bits[None] == 1, f[:, None], 1.0 - f[:, None]).prod(dim=2)
        inside = ((c >= 0) & (c < 16)).all(dim=2)
        ids = torch.where(inside, (c[..., 0] * 16 + c[..., 1]) * 16 + c[..., 2], -1)
    else:                            # distinct experts, some more popular; one pair in 16 over capacity, so dropped
        start = (e * torch.rand(n, 1, generator=g, device="cuda") ** 1.5).long().clamp_max(e - 1)
        hop = torch.randint(1, max(2, e // k), (n, 1), generator=g, device="cuda")
        ids = (start + hop * torch.arange(k, device="cuda")) % e
        w = torch.softmax(torch.randn(n, k, generator=g, device="cuda"), dim=1)
        ids = torch.where(torch.rand(n, k, generator=g, device="cuda") < 1.0 / 16, -1, ids)
    return ids.to(torch.int32).contiguous(), w.float().contiguous()


def _plan(ids, e):
    """Positions [n][k] of the pairs sorted by expert (-1: dropped)."""
    key = torch.where(ids < 0, e, ids).reshape(-1)
    order = torch.sort(key, stable=True)[1]
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return torch.where(ids < 0, -1, pos.reshape(ids.shape)).to(torch.int32).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, n, e = case["op"], case["n"], case["experts"]
    s = {"case": dict(case)}
    if op == "distill":
        k, t = case["k"], TYPES[case["dtype"]]
        s["student"] = torch.empty(n, e, device="cuda", dtype=t)
        step = max(1, (1 << 26) // e)
        for i in range(0, n, step):
            s["student"][i:i + step] = 2.5 * torch.randn(min(step, n - i), e, generator=g, device="cuda")
        s["teacher"] = torch.sort(3.0 * torch.randn(n, k, generator=g, device="cuda") + 4.0, dim=1, descending=True)[0].contiguous()
        start = torch.randint(0, e, (n, 1), generator=g, device="cuda")
        hop = torch.randint(1, max(2, e // k), (n, 1), generator=g, device="cuda")
        ids = ((start + hop * torch.arange(k, device="cuda")) % e).to(torch.int32)
        kept = torch.randint(0, k + 1, (n, 1), generator=g, device="cuda")
        short = torch.rand(n, 1, generator=g, device="cuda") < 0.25   # a quarter of the rows keep fewer, some none
        s["ids"] = torch.where(short & (torch.arange(k, device="cuda") >= kept), -1, ids).contiguous()
        s["scale"] = torch.rand(n, generator=g, device="cuda") + 0.5
        s["temperature"] = 2.0
        s["loss"] = torch.zeros(n, device="cuda")
        s["grad"] = torch.zeros(n, e, device="cuda", dtype=t) if case["grad"] else None
        return s
    if op in ("cells", "cells_backward"):
        d = torch.randn(n, 3, generator=g, device="cuda")
        if case["routing"] == "ray":
            a, b = _ball(2, g)
            x = a + (b - a) * ((torch.arange(n, device="cuda")[:, None] + 0.5) / n)
            d = (b - a).expand(n, 3)
        else:
            x = _ball(n, g)
        if case["routing"] == "gate":
            cell = (e * torch.rand(n, generator=g, device="cuda") ** 1.2).long().clamp_max(e - 1)
        else:
            c = ((x + 1.5) * (16.0 / 3.0)).long().clamp(0, 15)
            cell = (c[:, 0] * 16 + c[:, 1]) * 16 + c[:, 2]
        order = torch.sort(cell, stable=True)[1]
        count = torch.bincount(cell, minlength=e)
        s["x"], s["d"] = x[order].contiguous(), d[order].contiguous()
        s["offset"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.long), count.cumsum(0)]).to(torch.int32)
        s["longest"] = int(count.max())     # the plain form pads every cell's rows to it
        bound = torch.cat([torch.full((m,), (6.0 / (i + o)) ** 0.5) for m, i, o in
                           ((2048, 63, 32), (1056, 32, 32), (33, 32, 1), (180, 59, 3))])
        s["cell_w"] = ((2 * torch.rand(e, CELL_PARAMS, generator=g, device="cuda") - 1) * bound.cuda()).contiguous()
        s["out"] = torch.zeros(n, 4, device="cuda")
        s["hidden"] = torch.zeros(n, 64, device="cuda") if op == "cells_backward" or case["store"] else None
        if op == "cells_backward":
            _plain_cells(s)          # the forward pass that the gradient belongs to
            s["d_raw"] = torch.randn(n, 4, generator=g, device="cuda") / 64
            s["grad"] = torch.zeros(e, CELL_PARAMS, device="cuda")
        return s
    ids, w = _route(case, g)
    k = case["k"]
    if op == "sort":
        s["ids"] = ids
        s["offset"] = torch.zeros(e + 1, device="cuda", dtype=torch.int32)
        s["order"] = torch.full((n * k,), -1, device="cuda", dtype=torch.int32)
        s["pos"] = torch.zeros(n, k, device="cuda", dtype=torch.int32)
        return s
    t, c = TYPES[case["dtype"]], case["width"]

    def rows(m):
        return torch.randn(m, c, generator=g, device="cuda", dtype=torch.float32).to(t)

    s["pos"] = _plan(ids, e)
    s["weights"] = w if case["weighted"] else None
    if op == "dispatch":
        s["x"], s["rows"] = rows(n), torch.zeros(n * k, c, device="cuda", dtype=t)
    elif op == "combine":
        s["rows"], s["out"] = rows(n * k), torch.zeros(n, c, device="cuda", dtype=t)
    elif op == "dispatch_backward":
        s["d_rows"], s["x"], s["d_x"] = rows(n * k), rows(n), torch.zeros(n, c, device="cuda", dtype=t)
    else:
        s["d_out"], s["rows"], s["d_rows"] = rows(n), rows(n * k), torch.zeros(n * k, c, device="cuda", dtype=t)
    if op in ("dispatch_backward", "combine_backward"):
        s["d_weights"] = torch.zeros(n, k, device="cuda") if case["weighted"] else None
    return s


# ----------------------------------------------------------------- the operators, called

def _run_own(s):
    import neural_radiance_field_b200 as nb
    op = s["case"]["op"]
    if op == "sort":
        if "work" not in s:          # kept with the buffers, as a training loop does
            s["work"] = torch.empty(nb.nerf_expert_sort_workspace(*s["ids"].shape, s["case"]["experts"]), device="cuda", dtype=torch.uint8)
        nb.nerf_expert_sort(s["ids"], s["case"]["experts"], s["offset"], s["order"], s["pos"], s["work"])
        return {"offset": s["offset"], "order": s["order"], "pos": s["pos"]}
    if op == "dispatch":
        nb.nerf_expert_dispatch(s["x"], s["pos"], s["rows"], s["weights"])
        return {"rows": s["rows"]}
    if op == "combine":
        nb.nerf_expert_combine(s["rows"], s["pos"], s["out"], s["weights"])
        return {"out": s["out"]}
    if op == "dispatch_backward":
        nb.nerf_expert_dispatch_backward(s["d_rows"], s["x"], s["pos"], s["d_x"], s["weights"], s["d_weights"])
        return {"d_x": s["d_x"], "d_weights": s["d_weights"]}
    if op == "combine_backward":
        nb.nerf_expert_combine_backward(s["d_out"], s["rows"], s["pos"], s["d_rows"], s["weights"], s["d_weights"])
        return {"d_rows": s["d_rows"], "d_weights": s["d_weights"]}
    if op == "distill":
        nb.nerf_distill_topk(s["student"], s["teacher"], s["ids"], s["temperature"], s["loss"], s["grad"], s["scale"])
        return {"loss": s["loss"], "grad": s["grad"]}
    if op == "cells":
        nb.nerf_cells_forward(s["x"], s["d"], s["offset"], s["cell_w"], s["out"], s["hidden"])
        return {"raw": s["out"], "hidden": s["hidden"]}
    if "work" not in s:
        s["work"] = torch.empty(nb.nerf_cells_backward_workspace(s["case"]["n"], s["case"]["experts"]), device="cuda", dtype=torch.uint8)
    nb.nerf_cells_backward(s["x"], s["d"], s["offset"], s["cell_w"], s["hidden"], s["d_raw"], s["grad"], s["work"])
    return {"grad": s["grad"]}


# ----------------------------------------------------------------- the plain forms

def _pairs(s):
    """(kept pairs' positions, their point, their index in [n * k])."""
    pos = s["pos"].reshape(-1).long()
    at = (pos >= 0).nonzero()[:, 0]
    return pos[at], at // s["pos"].shape[1], at


def _plain_sort(s):
    e, ids = s["case"]["experts"], s["ids"].reshape(-1).long()
    key = torch.where(ids < 0, e, ids)
    by, order = torch.sort(key, stable=True)
    s["offset"].copy_(torch.searchsorted(by, torch.arange(e + 1, device=ids.device)))
    place = torch.arange(ids.numel(), device=ids.device)
    s["order"].copy_(torch.where(by < e, order, -1))
    pos = torch.empty_like(order)
    pos[order] = torch.where(by < e, place, -1)
    s["pos"].copy_(pos.reshape(s["pos"].shape))
    return {"offset": s["offset"], "order": s["order"], "pos": s["pos"]}


def _spread(x, s, out):
    """out[pos] = weight * x[point]."""
    to, point, at = _pairs(s)
    v = x.float()[point]
    if s["weights"] is not None:
        v = v * s["weights"].reshape(-1)[at][:, None]
    out[to] = v.to(out.dtype)


def _gathered(rows, s):
    """rows[pos] in fp32, [n][k][width], zero where a pair was dropped."""
    kept = s["pos"] >= 0
    v = rows.float()[s["pos"].long().clamp_min(0)]
    return torch.where(kept[..., None], v, 0.0), kept


def _folded(rows, s, out):
    """out[n] = sum over k of weight * rows[pos]."""
    v, kept = _gathered(rows, s)
    if s["weights"] is not None:
        v = v * torch.where(kept, s["weights"], 0.0)[..., None]
    out.copy_(v.sum(dim=1))


def _dots(rows, x, s):
    if s["d_weights"] is not None:
        s["d_weights"].copy_((_gathered(rows, s)[0] * x.float()[:, None]).sum(dim=2))
    return s["d_weights"]


def _plain_distill(s):
    t = s["temperature"]
    z = s["student"].float() / t
    m = z.max(dim=1, keepdim=True)[0]
    ex = torch.exp(z - m)
    total = ex.sum(dim=1, keepdim=True)
    kept = s["ids"] >= 0
    ids = s["ids"].long().clamp_min(0)
    y = torch.where(kept, s["teacher"] / t, float("-inf"))
    top = y.max(dim=1, keepdim=True)[0]
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(y - top)
    norm = p.sum(dim=1, keepdim=True)
    some = norm > 0
    p = p / torch.where(some, norm, 1.0)
    logp = y - top - torch.log(torch.where(some, norm, 1.0))
    logq = torch.gather(z, 1, ids) - m - torch.log(total)
    s["loss"].copy_(t * t * torch.where(kept, p * (logp - logq), 0.0).sum(dim=1))
    if s["grad"] is not None:
        gr = ex / total * some
        gr.scatter_add_(1, ids, -p)
        s["grad"].copy_(gr * (t * s["scale"])[:, None])
    return {"loss": s["loss"], "grad": s["grad"]}


def _encode(v, octaves):
    """[v, sin(2^k pi v), cos(2^k pi v)], coordinate-major blocks; the angles in 64 bits."""
    a = (v.double()[:, :, None] * (math.pi * 2.0 ** torch.arange(octaves, device=v.device, dtype=torch.float64))).reshape(v.shape[0], -1)
    return torch.cat([v, torch.sin(a).float(), torch.cos(a).float()], dim=1)


def _weights_of(w):
    e = w.shape[0]
    parts = torch.split(w, [2016, 32, 1024, 32, 32, 1, 177, 3], dim=1)
    return (parts[0].reshape(e, 32, 63), parts[1].reshape(e, 1, 32), parts[2].reshape(e, 32, 32), parts[3].reshape(e, 1, 32),
            parts[4].reshape(e, 1, 32), parts[5].reshape(e, 1, 1), parts[6].reshape(e, 3, 59), parts[7].reshape(e, 1, 3))


def _padding(s):
    """Row -> its place in [cell][longest], and the function that lays rows out so."""
    off, e, most = s["offset"].long(), s["offset"].numel() - 1, s["longest"]
    place = torch.arange(s["x"].shape[0], device=off.device)
    cell = torch.searchsorted(off, place, right=True) - 1
    slot = cell * most + place - off[cell]

    def padded(v):
        out = torch.zeros(e * most, v.shape[1], device=off.device)
        out[slot] = v
        return out.reshape(e, most, v.shape[1])

    return slot, padded


def _encodings(s):
    d = s["d"]
    return _encode(s["x"], 10), _encode(d / d.square().sum(dim=1, keepdim=True).sqrt(), 4)


def _plain_cells(s):
    w1, b1, w2, b2, ws, bs, wc, bc = _weights_of(s["cell_w"])
    slot, padded = _padding(s)
    px, pd = _encodings(s)
    h1 = torch.relu(torch.bmm(padded(px), w1.transpose(1, 2)) + b1)
    h2 = torch.relu(torch.bmm(h1, w2.transpose(1, 2)) + b2)
    rgb = torch.bmm(torch.cat([h2, padded(pd)], dim=2), wc.transpose(1, 2)) + bc
    s["out"].copy_(torch.cat([rgb, torch.bmm(h2, ws.transpose(1, 2)) + bs], dim=2).reshape(-1, 4)[slot])
    if s["hidden"] is not None:
        s["hidden"].copy_(torch.cat([h1, h2], dim=2).reshape(-1, 64)[slot])
    return {"raw": s["out"], "hidden": s["hidden"]}


def _plain_cells_backward(s):
    w2, ws, wc = (_weights_of(s["cell_w"])[i] for i in (2, 4, 6))
    _, padded = _padding(s)
    px, pd = _encodings(s)
    g, h = padded(s["d_raw"]), padded(s["hidden"])
    h1, h2, gc, gs = h[:, :, :32], h[:, :, 32:], g[:, :, :3], g[:, :, 3:]
    g2 = (torch.bmm(gc, wc[:, :, :32]) + gs * ws) * (h2 > 0)
    g1 = torch.bmm(g2, w2) * (h1 > 0)
    both = torch.cat([h2, padded(pd)], dim=2)
    parts = [torch.bmm(g1.transpose(1, 2), padded(px)), g1.sum(dim=1), torch.bmm(g2.transpose(1, 2), h1), g2.sum(dim=1),
             torch.bmm(gs.transpose(1, 2), h2), gs.sum(dim=1), torch.bmm(gc.transpose(1, 2), both), gc.sum(dim=1)]
    s["grad"].copy_(torch.cat([v.reshape(v.shape[0], -1) for v in parts], dim=1))
    return {"grad": s["grad"]}


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "sort":
        return _plain_sort(s)
    if op == "dispatch":
        _spread(s["x"], s, s["rows"])
        return {"rows": s["rows"]}
    if op == "combine":
        _folded(s["rows"], s, s["out"])
        return {"out": s["out"]}
    if op == "dispatch_backward":
        _folded(s["d_rows"], s, s["d_x"])
        return {"d_x": s["d_x"], "d_weights": _dots(s["d_rows"], s["x"], s)}
    if op == "combine_backward":
        _spread(s["d_out"], s, s["d_rows"])
        return {"d_rows": s["d_rows"], "d_weights": _dots(s["rows"], s["d_out"], s)}
    if op == "distill":
        return _plain_distill(s)
    return _plain_cells(s) if op == "cells" else _plain_cells_backward(s)


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, n, e = case["op"], case["n"], case["experts"]
    if op == "distill":
        size, k, g = 4 if case["dtype"] == "fp32" else 2, case["k"], case["grad"]
        return {"bytes": n * e * size * (2 if g else 1) + n * k * 8 + n * (8 if g else 4), "flops": n * e * (6 if g else 4)}
    if op == "cells":
        return {"bytes": n * (296 if case["store"] else 40) + 4 * e + 4 * CELL_PARAMS * min(e, n), "flops": 2 * 3249 * n}
    if op == "cells_backward":
        # h2's and h1's gradients and every weight's; of the weights the backward reads W2 and the heads on h2
        return {"bytes": n * 296 + 4 * e + 4 * (1152 * min(e, n) + CELL_PARAMS * e), "flops": 2 * (128 + 1024 + 3249) * n}
    k = case["k"]
    if op == "sort":
        return {"bytes": 12 * n * k + 4 * e, "flops": n * k}
    kept = n * k * (15.0 / 16 if case["routing"] == "gate" else 0.9)
    size, c, w = 4 if case["dtype"] == "fp32" else 2, case["width"], 4 * n * k if case["weighted"] else 0
    b = size * c * (n + kept) + 4 * n * k + w
    if op == "combine_backward":
        return {"bytes": b + (size * c * kept + 4 * n * k if w else 0), "flops": (3 if w else 1) * c * kept}
    if op == "dispatch_backward":
        return {"bytes": b + (size * c * n + 4 * n * k if w else 0), "flops": (4 if w else 2) * c * kept}
    return {"bytes": b, "flops": 2 * c * kept}


# ----------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, n, e = case["op"], case["n"], case["experts"]
    if op == "sort":
        ids = s["ids"].cpu().numpy().reshape(-1)
        kept = np.flatnonzero((ids >= 0) & (ids < e))
        by = kept[np.argsort(ids[kept], kind="stable")]
        order = np.full(ids.size, -1, np.int32)
        order[:by.size] = by
        pos = np.full(ids.size, -1, np.int32)
        pos[by] = np.arange(by.size)
        offset = np.concatenate([[0], np.cumsum(np.bincount(ids[kept], minlength=e))]).astype(np.int32)
        return {"offset": offset, "order": order, "pos": pos.reshape(s["pos"].shape)}
    if op == "distill":
        if n * e > 300_000_000:
            return None
        loss = torch.zeros(n, dtype=torch.float64, device="cuda")
        grad = torch.zeros(n, e, dtype=torch.float64, device="cuda") if case["grad"] else None
        t, step = s["temperature"], max(1, 20_000_000 // e)
        for i in range(0, n, step):
            j = min(n, i + step)
            logq = torch.log_softmax(s["student"][i:j].double() / t, dim=1)
            teacher = torch.full((j - i, e + 1), -math.inf, dtype=torch.float64, device="cuda")
            ids = s["ids"][i:j].long()
            teacher.scatter_(1, torch.where(ids < 0, e, ids), s["teacher"][i:j].double() / t)
            teacher[:, e] = -math.inf
            teacher = teacher[:, :e]
            empty = (ids < 0).all(dim=1)
            logp = torch.where(empty[:, None], 0.0, torch.log_softmax(teacher, dim=1))
            p = torch.where(empty[:, None], 0.0, torch.exp(logp))
            loss[i:j] = t * t * torch.where(p > 0, p * (logp - logq), 0.0).sum(dim=1)
            if grad is not None:
                full = t * s["scale"][i:j, None].double() * (torch.exp(logq) - p)
                grad[i:j] = torch.where(empty[:, None], 0.0, full)
        return {"loss": loss, "grad": grad}
    if op in ("cells", "cells_backward"):
        off, w = s["offset"].tolist(), s["cell_w"].double()
        x, d = s["x"].double(), s["d"].double()
        d = d / torch.linalg.norm(d, dim=1, keepdim=True)

        def gamma(v, octaves):
            cols = [f(math.pi * 2.0 ** k * v[:, c]) for f in (torch.sin, torch.cos) for c in range(3) for k in range(octaves)]
            return torch.cat([v, torch.stack(cols, dim=1)], dim=1)

        px, pd = gamma(x, 10), gamma(d, 4)
        raw = torch.zeros(n, 4, dtype=torch.float64, device="cuda")
        hidden = torch.zeros(n, 64, dtype=torch.float64, device="cuda")
        grad = torch.zeros(e, CELL_PARAMS, dtype=torch.float64, device="cuda")
        for c in range(e):
            a, b = off[c], off[c + 1]
            if a == b:
                continue
            p = torch.tensor_split(w[c], np.cumsum([2016, 32, 1024, 32, 32, 1, 177]).tolist())
            if op == "cells":
                h1 = (px[a:b] @ p[0].view(32, 63).T + p[1]).clamp_min(0)
                h2 = (h1 @ p[2].view(32, 32).T + p[3]).clamp_min(0)
                hidden[a:b] = torch.cat([h1, h2], dim=1)
            else:
                h1, h2 = s["hidden"][a:b].double().split(32, dim=1)
            both = torch.cat([h2, pd[a:b]], dim=1)
            if op == "cells":
                raw[a:b, :3] = both @ p[6].view(3, 59).T + p[7]
                raw[a:b, 3] = h2 @ p[4] + p[5]
                continue
            g = s["d_raw"][a:b].double()
            z2 = (g[:, :3] @ p[6].view(3, 59)[:, :32] + g[:, 3:] * p[4]) * (h2 > 0)
            z1 = (z2 @ p[2].view(32, 32)) * (h1 > 0)
            grad[c] = torch.cat([(z1.T @ px[a:b]).reshape(-1), z1.sum(0), (z2.T @ h1).reshape(-1), z2.sum(0), g[:, 3] @ h2,
                                 g[:, 3].sum().view(1), (g[:, :3].T @ both).reshape(-1), g[:, :3].sum(0)])
        if op == "cells":
            return {"raw": raw, "hidden": hidden if case["store"] else None}
        return {"grad": grad}
    pos, k = s["pos"].long(), case["k"]
    w = s["weights"].double() if s["weights"] is not None else torch.ones(n, k, dtype=torch.float64, device="cuda")

    def to_rows(v, rows):
        out = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            on = pos[:, j] >= 0
            out[pos[on, j]] = v.double()[on] * w[on, j, None]
        return out

    def to_points(rows, v):
        out = torch.zeros(n, case["width"], dtype=torch.float64, device="cuda")
        dots = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            on = pos[:, j] >= 0
            taken = rows[pos[on, j]].double()
            out[on] += taken * w[on, j, None]
            if v is not None:
                dots[on, j] = (taken * v[on].double()).sum(dim=1)
        return out, dots

    if op == "dispatch":
        return {"rows": to_rows(s["x"], s["rows"])}
    if op == "combine":
        return {"out": to_points(s["rows"], None)[0]}
    if op == "dispatch_backward":
        d_x, d_w = to_points(s["d_rows"], s["x"])
        return {"d_x": d_x, "d_weights": d_w if case["weighted"] else None}
    d_w = to_points(s["rows"], s["d_out"])[1] if case["weighted"] else None
    return {"d_rows": to_rows(s["d_out"], s["rows"]), "d_weights": d_w}
