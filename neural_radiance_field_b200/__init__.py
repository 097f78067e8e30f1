"""B200 forward NeRF renderer: a thin Python binding over libnerf.so.

Every function here only marshals torch tensors (device memory, the current
CUDA stream) into the C ABI of include/nerf.h; all the work runs in the
library's CUDA kernels. Importing this package does not load the library;
the first call does, and fails loudly when it is missing.
"""
from __future__ import annotations

import ctypes

from . import _capi
from ._capi import (NERF_BF16, NERF_DTYPE_BF16, NERF_DTYPE_FP16, NERF_DTYPE_FP32, NERF_FP32,
                    NERF_LAST_1E10, NERF_LAST_TO_FAR, NERF_MODEL_HASHGRID, NERF_MODEL_KILONERF,
                    NERF_MODEL_MLP, NERF_SIGMA_RELU, NERF_SIGMA_SOFTPLUS, NERF_TF32,
                    NerfError, nerf_config, nerf_params)

__all__ = ["Renderer", "nerf_raygen", "nerf_raygen_batch", "nerf_hash_encode_backward",
           "nerf_expert_sort_workspace", "nerf_expert_sort", "nerf_expert_dispatch",
           "nerf_expert_dispatch_backward", "nerf_expert_combine", "nerf_expert_combine_backward",
           "nerf_distill_topk", "nerf_cells_forward", "nerf_cells_backward_workspace",
           "nerf_cells_backward", "nerf_test_stratified", "nerf_test_pe",
           "nerf_test_composite", "nerf_test_sample_pdf", "NerfError", "nerf_config",
           "nerf_params"]


def _ptr(t):
    if t is None:
        return None
    import torch
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _hptr(t):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("expected a contiguous host tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def nerf_raygen(H, W, focal, c2w, rays_o, rays_d, stream=None):
    """c2w: 12 host floats (sequence or array); rays_o, rays_d: CUDA [H*W, 3]."""
    c = (ctypes.c_float * 12)(*[float(v) for v in list(c2w)])
    _capi.check(_capi.lib().nerf_raygen(int(H), int(W), float(focal), c, _ptr(rays_o),
                                        _ptr(rays_d), _stream(stream)))


def nerf_raygen_batch(H, W, focal, c2ws, rays_o, rays_d, stream=None):
    """c2ws: n_cams x 12 host floats; rays_o, rays_d: CUDA [n_cams*H*W, 3], camera-major."""
    flat = [float(v) for cam in c2ws for v in list(cam)]
    n_cams = len(flat) // 12
    if n_cams * 12 != len(flat):
        raise ValueError("each camera needs 12 values ([3][4] row-major)")
    c = (ctypes.c_float * len(flat))(*flat)
    _capi.check(_capi.lib().nerf_raygen_batch(int(H), int(W), float(focal), n_cams, c,
                                              _ptr(rays_o), _ptr(rays_d), _stream(stream)))


def nerf_test_stratified(rays_o, rays_d, near, far, n, seed, perturb, out_t, out_x=None,
                         stream=None):
    _capi.check(_capi.lib().nerf_test_stratified(
        _ptr(rays_o), _ptr(rays_d), rays_o.shape[0], float(near), float(far), int(n), int(seed),
        int(perturb), _ptr(out_t), _ptr(out_x), _stream(stream)))


def nerf_test_pe(x, L, out, stream=None):
    _capi.check(_capi.lib().nerf_test_pe(_ptr(x), x.shape[0], int(L), _ptr(out), _stream(stream)))


def nerf_test_composite(raw, t, rays_d, far, last_delta_mode, march_step, sigma_act, white_bkgd,
                        out_rgb, out_depth, out_acc, out_weights=None, stream=None):
    R, S = t.shape
    _capi.check(_capi.lib().nerf_test_composite(
        _ptr(raw), _ptr(t), _ptr(rays_d), R, S, float(far), int(last_delta_mode),
        float(march_step), int(sigma_act), int(white_bkgd), _ptr(out_rgb), _ptr(out_depth),
        _ptr(out_acc), _ptr(out_weights), _stream(stream)))


def nerf_test_sample_pdf(t_coarse, weights, n_fine, seed, perturb, out_t_fine=None,
                         out_below=None, out_t_all=None, stream=None):
    R, Nc = t_coarse.shape
    _capi.check(_capi.lib().nerf_test_sample_pdf(
        _ptr(t_coarse), _ptr(weights), R, Nc, int(n_fine), int(seed), int(perturb),
        _ptr(out_t_fine), _ptr(out_below), _ptr(out_t_all), _stream(stream)))


def nerf_test_march(rays_o, rays_d, near, step, K, occupancy, out_count, out_live=None,
                    stream=None):
    _capi.check(_capi.lib().nerf_test_march(
        _ptr(rays_o), _ptr(rays_d), rays_o.shape[0], float(near), float(step), int(K),
        _ptr(occupancy), _ptr(out_count), _ptr(out_live), _stream(stream)))


def nerf_test_route_cells(x, out_cell, out_cell_count, out_cell_offset, out_order=None,
                          stream=None):
    _capi.check(_capi.lib().nerf_test_route_cells(
        _ptr(x), x.shape[0], _ptr(out_cell), _ptr(out_cell_count), _ptr(out_cell_offset),
        _ptr(out_order), _stream(stream)))


def nerf_test_hash_encode(x, hash_table, out_feat, out_rows=None, stream=None):
    _capi.check(_capi.lib().nerf_test_hash_encode(
        _ptr(x), x.shape[0], _ptr(hash_table), _ptr(out_feat), _ptr(out_rows), _stream(stream)))


def nerf_hash_encode_backward(x, d_feat, grad_table, deterministic=False, stream=None):
    """Scatter-add of encoding gradients into grad_table (accumulated); see the header."""
    _capi.check(_capi.lib().nerf_hash_encode_backward(_ptr(x), x.shape[0], _ptr(d_feat),
                                                      _ptr(grad_table), int(bool(deterministic)),
                                                      _stream(stream)))


def nerf_test_sh(d, out, stream=None):
    _capi.check(_capi.lib().nerf_test_sh(_ptr(d), d.shape[0], _ptr(out), _stream(stream)))


def _current(name, t):
    """The device of an operator's first tensor, which has to be the current one (the C
    ABI works on that)."""
    import torch
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on cuda:{dev}, which is not the current device")
    return dev


def _arg(name, t, dtype, shape, dev):
    """Address of a tensor argument: contiguous, of the given type and shape, on device `dev`."""
    try:
        if t.dtype is not dtype or t.shape != shape:
            raise ValueError(f"{name}: expected {dtype} of shape {tuple(shape)}, got {t.dtype} of {tuple(t.shape)}")
        if t.get_device() != dev:
            raise ValueError(f"{name}: expected a CUDA tensor on the current device (cuda:{dev}), got one on {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
        return t.data_ptr()
    except AttributeError:
        raise ValueError(f"{name}: expected a CUDA tensor, got {type(t).__name__}") from None


def _opt(name, t, dtype, shape, dev):
    return None if t is None else _arg(name, t, dtype, shape, dev)


_DTYPE_CODES = {}


def _rows_dtype(name, t):
    """(torch dtype, NERF_DTYPE_*) of a row tensor."""
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.float32: NERF_DTYPE_FP32, torch.bfloat16: NERF_DTYPE_BF16,
                             torch.float16: NERF_DTYPE_FP16})
    code = _DTYPE_CODES.get(getattr(t, "dtype", None))
    if code is None:
        raise ValueError(f"{name}: expected a float32, bfloat16 or float16 tensor")
    return t.dtype, code


def _size(name, v, bits=32):
    """A size as the C ABI's signed integer of `bits` bits, which ctypes would cut to them unasked."""
    v = int(v)
    if not -(1 << bits - 1) <= v < 1 << bits - 1:
        raise ValueError(f"{name}: {v} does not fit {bits} bits")
    return v


def _shape2(name, t):
    """Sizes of a tensor of two dimensions, the second (a C int) below 2^31."""
    s = getattr(t, "shape", ())
    if len(s) != 2:
        raise ValueError(f"{name}: expected a tensor of 2 dimensions")
    if s[1] >= 1 << 31:
        raise ValueError(f"{name}: {s[1]} columns do not fit 32 bits")
    return s


def _work(t, dev):
    if not hasattr(t, "element_size"):
        raise ValueError("workspace: expected a CUDA tensor")
    return _arg("workspace", t, t.dtype, t.shape, dev), t.numel() * t.element_size()


def _call(fn, *args, stream, dev):
    """The library call on `stream`, else on the current stream's raw handle (building
    torch's Stream object for it would take a third of a small call's time)."""
    import torch
    s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)
    lib = _capi._lib or _capi.lib()
    status = getattr(lib, fn)(*args, s)
    if status:
        _capi.check(status)


def nerf_expert_sort_workspace(n, k, n_experts):
    """Bytes of workspace that nerf_expert_sort needs."""
    b = ctypes.c_int64()
    _capi.check(_capi.lib().nerf_expert_sort_workspace(_size("n", n, 64), _size("k", k), _size("n_experts", n_experts),
                                                        ctypes.byref(b)))
    return b.value


def nerf_expert_sort(ids, n_experts, out_offset, out_order, out_pos, workspace, stream=None):
    """Stable sort of (point, expert) pairs by expert; ids [n, k] int32, out_order [n * k]
    or None; workspace: any tensor of at least nerf_expert_sort_workspace bytes."""
    import torch
    n, k = _shape2("ids", ids)
    e = _size("n_experts", n_experts)
    i32, dev = torch.int32, _current("ids", ids)
    _call("nerf_expert_sort", _arg("ids", ids, i32, (n, k), dev), n, k, e,
          _arg("out_offset", out_offset, i32, (e + 1,), dev), _opt("out_order", out_order, i32, (n * k,), dev),
          _arg("out_pos", out_pos, i32, (n, k), dev), *_work(workspace, dev), stream=stream, dev=dev)


def nerf_expert_dispatch(x, pos, rows, weights=None, stream=None):
    """rows[pos[i, j]] = weights[i, j] * x[i]; x [n, width], pos [n, k], rows [n * k, width]."""
    import torch
    (n, c), k = _shape2("x", x), _shape2("pos", pos)[1]
    (t, code), dev = _rows_dtype("x", x), _current("x", x)
    _call("nerf_expert_dispatch", _arg("x", x, t, (n, c), dev), code, n, c,
          _arg("pos", pos, torch.int32, (n, k), dev), k,
          _opt("weights", weights, torch.float32, (n, k), dev), _arg("rows", rows, t, (n * k, c), dev),
          stream=stream, dev=dev)


def nerf_expert_dispatch_backward(d_rows, x, pos, d_x, weights=None, d_weights=None, stream=None):
    """d_x and d_weights of nerf_expert_dispatch (either may be None); see the header."""
    import torch
    c, (n, k) = _shape2("d_rows", d_rows)[1], _shape2("pos", pos)
    (t, code), dev, f32 = _rows_dtype("d_rows", d_rows), _current("d_rows", d_rows), torch.float32
    _call("nerf_expert_dispatch_backward", _arg("d_rows", d_rows, t, (n * k, c), dev),
          _opt("x", x, t, (n, c), dev), code, n, c, _arg("pos", pos, torch.int32, (n, k), dev), k,
          _opt("weights", weights, f32, (n, k), dev), _opt("d_x", d_x, t, (n, c), dev),
          _opt("d_weights", d_weights, f32, (n, k), dev), stream=stream, dev=dev)


def nerf_expert_combine(rows, pos, out, weights=None, stream=None):
    """out[i] = sum_j weights[i, j] * rows[pos[i, j]]; rows [n * k, width], out [n, width]."""
    import torch
    c, (n, k) = _shape2("rows", rows)[1], _shape2("pos", pos)
    (t, code), dev = _rows_dtype("rows", rows), _current("rows", rows)
    _call("nerf_expert_combine", _arg("rows", rows, t, (n * k, c), dev), code, n, c,
          _arg("pos", pos, torch.int32, (n, k), dev), k,
          _opt("weights", weights, torch.float32, (n, k), dev), _arg("out", out, t, (n, c), dev),
          stream=stream, dev=dev)


def nerf_expert_combine_backward(d_out, rows, pos, d_rows, weights=None, d_weights=None,
                                 stream=None):
    """d_rows and d_weights of nerf_expert_combine (either may be None); see the header."""
    import torch
    (n, c), k = _shape2("d_out", d_out), _shape2("pos", pos)[1]
    (t, code), dev, f32 = _rows_dtype("d_out", d_out), _current("d_out", d_out), torch.float32
    _call("nerf_expert_combine_backward", _arg("d_out", d_out, t, (n, c), dev),
          _opt("rows", rows, t, (n * k, c), dev), code, n, c, _arg("pos", pos, torch.int32, (n, k), dev), k,
          _opt("weights", weights, f32, (n, k), dev), _opt("d_rows", d_rows, t, (n * k, c), dev),
          _opt("d_weights", d_weights, f32, (n, k), dev), stream=stream, dev=dev)


def nerf_distill_topk(student, teacher_logits, teacher_ids, temperature, out_loss, out_grad=None,
                      row_scale=None, stream=None):
    """Distillation loss [n] (and gradient [n, classes]) of student logits [n, classes]
    against a teacher's kept logits and ids [n, k]; see the header."""
    import torch
    (n, e), k = _shape2("student", student), _shape2("teacher_ids", teacher_ids)[1]
    (t, code), dev, f32 = _rows_dtype("student", student), _current("student", student), torch.float32
    _call("nerf_distill_topk", _arg("student", student, t, (n, e), dev), code, n, e,
          _arg("teacher_logits", teacher_logits, f32, (n, k), dev),
          _arg("teacher_ids", teacher_ids, torch.int32, (n, k), dev), k, float(temperature),
          _opt("row_scale", row_scale, f32, (n,), dev), _arg("out_loss", out_loss, f32, (n,), dev),
          _opt("out_grad", out_grad, t, (n, e), dev), stream=stream, dev=dev)


def nerf_cells_forward(x, d, offset, cell_w, out_raw, out_hidden=None, stream=None):
    """Per-cell networks on rows sorted by cell: out_raw [n, 4], out_hidden [n, 64] or None."""
    import torch
    n, e = _shape2("x", x)[0], _size("n_cells", _shape2("cell_w", cell_w)[0])
    f32, dev = torch.float32, _current("x", x)
    _call("nerf_cells_forward", _arg("x", x, f32, (n, 3), dev), _arg("d", d, f32, (n, 3), dev), n,
          _arg("offset", offset, torch.int32, (e + 1,), dev), e,
          _arg("cell_w", cell_w, f32, (e, 3317), dev), _arg("out_raw", out_raw, f32, (n, 4), dev),
          _opt("out_hidden", out_hidden, f32, (n, 64), dev), stream=stream, dev=dev)


def nerf_cells_backward_workspace(n_rows, n_cells):
    """Bytes of workspace that nerf_cells_backward needs."""
    b = ctypes.c_int64()
    _capi.check(_capi.lib().nerf_cells_backward_workspace(_size("n_rows", n_rows, 64), _size("n_cells", n_cells), ctypes.byref(b)))
    return b.value


def nerf_cells_backward(x, d, offset, cell_w, hidden, d_raw, grad_cell_w, workspace, stream=None):
    """Weight gradient of nerf_cells_forward (overwritten), from its hidden layers."""
    import torch
    n, e = _shape2("x", x)[0], _size("n_cells", _shape2("cell_w", cell_w)[0])
    f32, dev = torch.float32, _current("x", x)
    _call("nerf_cells_backward", _arg("x", x, f32, (n, 3), dev), _arg("d", d, f32, (n, 3), dev), n,
          _arg("offset", offset, torch.int32, (e + 1,), dev), e,
          _arg("cell_w", cell_w, f32, (e, 3317), dev), _arg("hidden", hidden, f32, (n, 64), dev),
          _arg("d_raw", d_raw, f32, (n, 4), dev),
          _arg("grad_cell_w", grad_cell_w, f32, (e, 3317), dev), *_work(workspace, dev), stream=stream, dev=dev)


class Renderer:
    """Owns a nerf_ctx (nerf_create / nerf_destroy). The arguments are the fields
    of nerf_config (include/nerf.h): precision NERF_FP32 (fused CUDA-core
    network), NERF_BF16 (the 8x256 network on the tensor cores with bf16
    weights) or NERF_TF32 (fp32 weights, the layers on the tensor cores as
    three tf32 products each, at fp32-level accuracy; W of 128 or 256)."""

    def __init__(self, model=NERF_MODEL_MLP, D=8, W=256, skip=4, L_pos=10, L_dir=4,
                 sigma_act=NERF_SIGMA_RELU, precision=NERF_FP32, last_delta_mode=NERF_LAST_1E10,
                 white_bkgd=0, max_rays=1 << 16, max_samples=192):
        self.cfg = nerf_config(model, D, W, skip, L_pos, L_dir, sigma_act, precision,
                               last_delta_mode, white_bkgd, max_rays, max_samples)
        h = ctypes.c_void_p()
        _capi.check(_capi.lib().nerf_create(ctypes.byref(self.cfg), ctypes.byref(h)))
        self.ctx = h

    def close(self):
        if getattr(self, "ctx", None):
            _capi.lib().nerf_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @staticmethod
    def params(coarse_w=None, fine_w=None, occupancy=None, cell_w=None, hash_table=None,
               hash_mlp=None, march_step=0.0, ert_T=0.0, seed=0, perturb=1):
        """A nerf_params holding the device pointers of the given tensors. The
        library reads the tensors through these pointers on every call, so the
        returned object keeps references to them: they stay allocated for as long
        as it is alive, and a temporary passed here cannot be freed and its
        memory reused while the params are in use."""
        p = nerf_params()
        p._tensors = tuple(t for t in (coarse_w, fine_w, occupancy, cell_w, hash_table, hash_mlp)
                           if t is not None)
        p.coarse_w = coarse_w.data_ptr() if coarse_w is not None else None
        p.fine_w = fine_w.data_ptr() if fine_w is not None else None
        p.occupancy = occupancy.data_ptr() if occupancy is not None else None
        p.cell_w = cell_w.data_ptr() if cell_w is not None else None
        p.hash_table = hash_table.data_ptr() if hash_table is not None else None
        p.hash_mlp = hash_mlp.data_ptr() if hash_mlp is not None else None
        p.march_step = march_step
        p.ert_T = ert_T
        p.seed = seed
        p.perturb = perturb
        return p

    def render(self, rays_o, rays_d, near, far, n_coarse, n_fine, params, out_rgb, out_depth,
               out_acc, stream=None):
        _capi.check(_capi.lib().nerf_render(
            self.ctx, _ptr(rays_o), _ptr(rays_d), rays_o.shape[0], float(near), float(far),
            int(n_coarse), int(n_fine), ctypes.byref(params), _ptr(out_rgb), _ptr(out_depth),
            _ptr(out_acc), _stream(stream)), self.ctx)

    def render_trace(self, rays_o, rays_d, near, far, n_coarse, n_fine, params, out_rgb,
                     out_depth, out_acc, raw_coarse=None, w_coarse=None, t_fine=None, below=None,
                     t_all=None, raw_fine=None, stream=None):
        """nerf_render that also copies the render's intermediates into the given
        CUDA tensors (any may be None); see nerf_render_trace."""
        tr = _capi.nerf_trace(*[t.data_ptr() if t is not None else None for t in
                                (raw_coarse, w_coarse, t_fine, below, t_all, raw_fine)])
        for t in (raw_coarse, w_coarse, t_fine, below, t_all, raw_fine):
            _ptr(t)                                       # device and contiguous
        _capi.check(_capi.lib().nerf_render_trace(
            self.ctx, _ptr(rays_o), _ptr(rays_d), rays_o.shape[0], float(near), float(far),
            int(n_coarse), int(n_fine), ctypes.byref(params), _ptr(out_rgb), _ptr(out_depth),
            _ptr(out_acc), ctypes.byref(tr), _stream(stream)), self.ctx)

    def loss_grad(self, rays_o, rays_d, near, far, n_coarse, n_fine, params, target_rgb,
                  out_loss, grad_coarse, grad_fine=None, stream=None):
        """Training-step loss and gradients (fp32 contexts); see nerf_loss_grad."""
        _capi.check(_capi.lib().nerf_loss_grad(
            self.ctx, _ptr(rays_o), _ptr(rays_d), rays_o.shape[0], float(near), float(far),
            int(n_coarse), int(n_fine), ctypes.byref(params), _ptr(target_rgb), _ptr(out_loss),
            _ptr(grad_coarse), _ptr(grad_fine), _stream(stream)), self.ctx)

    def render_host(self, rays_o, rays_d, near, far, n_coarse, n_fine, params, out_rgb, out_depth,
                    out_acc, stream=None):
        _capi.check(_capi.lib().nerf_render_host(
            self.ctx, _hptr(rays_o), _hptr(rays_d), rays_o.shape[0], float(near), float(far),
            int(n_coarse), int(n_fine), ctypes.byref(params), _hptr(out_rgb), _hptr(out_depth),
            _hptr(out_acc), _stream(stream)), self.ctx)

    def test_mlp(self, weights, x, d, out_raw, stream=None):
        _capi.check(_capi.lib().nerf_test_mlp(self.ctx, _ptr(weights), _ptr(x), _ptr(d),
                                              x.shape[0], _ptr(out_raw), _stream(stream)),
                    self.ctx)

    def timing_enable(self, enable=True):
        _capi.check(_capi.lib().nerf_timing_enable(self.ctx, int(enable)), self.ctx)

    def timing_read(self):
        """(summed network-kernel ms, number of timed launches) since the last read."""
        ms = ctypes.c_double()
        n = ctypes.c_int64()
        _capi.check(_capi.lib().nerf_timing_read(self.ctx, ctypes.byref(ms), ctypes.byref(n)),
                    self.ctx)
        return ms.value, n.value

    def timing_read_kinds(self):
        """{kernel class: (summed ms, launches)} since the last read, for every
        class of nerf_timing_read_kinds."""
        n = len(_capi.TIMED_KINDS)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        _capi.check(_capi.lib().nerf_timing_read_kinds(self.ctx, ms, cnt), self.ctx)
        return {k: (ms[i], cnt[i]) for i, k in enumerate(_capi.TIMED_KINDS)}

    def sync_status(self, stream=None):
        _capi.check(_capi.lib().nerf_sync_status(self.ctx, _stream(stream)), self.ctx)
