"""Python binding of the operators around attention: the sum and norm between two
blocks and dense layers on tokens (include/imgstencil.h).

Tensors are torch device tensors n x len x c with a contiguous last dimension and
any other strides; an fp16 NHWC feature map (n, H, W, C) viewed as (n, H * W, C) is
one, and so is a token tensor n x len x heads x d viewed with its heads joined. The
functions with the C names marshal arguments to the C ABI and nothing else; BlockNorm
and Dense check their tensors and launch on torch's current stream of the tensors'
device.
"""
import ctypes

from . import _abi
from ._abi import block_norm_desc, conv2d_plan_info, dense_desc, is_rows
from .attention import (_ALLOCATED, _INT_MAX, _NORMS, _Layouts, _check_device, _check_weight, _device_calls, _dtype,
                        _one_device, _ptr, _sig, _steps)

_ACTIVATIONS = {"none": _abi.IS_ACT_NONE, "relu": _abi.IS_ACT_RELU, "gelu": _abi.IS_ACT_GELU,
                "gelu_tanh": _abi.IS_ACT_GELU_TANH, "silu": _abi.IS_ACT_SILU}


# ------------------------------------------------------------------ the C names
def block_norm_forward(desc, x_ptr, y_ptr, gate_ptr, post_weight_ptr, weight_ptr, bias_ptr, scale_ptr, shift_ptr,
                       x_out_ptr, out_ptr, stream):
    """Raw pointers (ints, 0 or None where absent) and a hipStream_t (int)."""
    _abi.check(_abi.load().block_norm_forward(ctypes.byref(desc), x_ptr or None, y_ptr or None, gate_ptr or None,
                                              post_weight_ptr or None, weight_ptr or None, bias_ptr or None,
                                              scale_ptr or None, shift_ptr or None, x_out_ptr or None, out_ptr or None,
                                              stream or None), "block_norm_forward")


def dense_create(desc):
    """Returns an opaque plan handle (int); raises ImgStencilError on a bad desc."""
    plan = ctypes.c_void_p()
    _abi.check(_abi.load().dense_create(ctypes.byref(desc), ctypes.byref(plan)), "dense_create")
    return plan.value


def dense_destroy(plan):
    _abi.load().dense_destroy(plan)


def dense_workspace_size(plan):
    n = ctypes.c_size_t()
    _abi.check(_abi.load().dense_workspace_size(plan, ctypes.byref(n)), "dense_workspace_size")
    return n.value


def dense_get_plan_info(plan):
    """grid: (tiles of all entries, parts of the inner sum, 1); tile: (features, rows).
    is_k13_dense_few has a workgroup for every tile; those of is_k13_dense, as many as
    the device holds at a time, walk the tiles of all parts."""
    info = conv2d_plan_info()
    _abi.check(_abi.load().dense_get_plan_info(plan, ctypes.byref(info)), "dense_get_plan_info")
    return {"kernel": info.kernel.decode(), "grid": (info.grid_x, info.grid_y, info.grid_z), "block": info.block,
            "lds_bytes": info.lds_bytes, "tile": (info.tile_w, info.tile_h), "flops": info.flops, "bytes": info.bytes}


def dense_forward(plan, x_ptr, w_ptr, bias_ptr, residual_ptr, out_ptr, ws_ptr, ws_bytes, stream):
    _abi.check(_abi.load().dense_forward(plan, x_ptr or None, w_ptr or None, bias_ptr or None, residual_ptr or None,
                                         out_ptr or None, ws_ptr or None, ws_bytes, stream or None), "dense_forward")


# ---------------------------------------------------------------- torch helpers
def _check_rows(t, name, dtype, c=None, shape=None):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError("%s must be a %s tensor" % (name, dtype))
    if t.dim() != 3:
        raise ValueError("%s must be n x len x c, got shape %s" % (name, tuple(t.shape)))
    if max(t.shape) > _INT_MAX:
        raise ValueError("%s has a dimension over %d, got shape %s" % (name, _INT_MAX, tuple(t.shape)))
    if c is not None and t.shape[2] != c:
        raise ValueError("%s has %d channels, expected %d" % (name, t.shape[2], c))
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)


def _rows(t, dense=False):
    """The row tensor t, or a new dense one of its shape."""
    n, length, c = t.shape
    return is_rows(n, length, length * c if dense else t.stride(0), c if dense else t.stride(1))


def _check_per_entry(t, name, x):
    """(n or 1) x c of x's dtype; returns the stride between entries (0: one row)."""
    import torch
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype != x.dtype:
        raise TypeError("%s must be a %s tensor" % (name, x.dtype))
    if t.dim() != 2 or t.shape[0] not in (1, x.shape[0]) or t.shape[1] != x.shape[2]:
        raise ValueError("%s must be %d (or 1) x %d, got shape %s" % (name, x.shape[0], x.shape[2], tuple(t.shape)))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    return 0 if t.shape[0] == 1 else t.stride(0)


class BlockNorm:
    """The sum and norm between two blocks, for rows of c channels:

        x_out = x + residual_scale * gate * post(y)
        out   = norm(x_out) * weight * (1 + scale) + shift + bias

    (The bias is not scaled. A norm with weight and bias that is modulated afterwards,
    (norm(x_out) * weight + bias) * (1 + scale) + shift, is had without bias and with
    shift + bias * (1 + scale), rounded to its type, as the shift.)

    norm: "rms", "layer" or None (the sum alone); post: "rms", "layer" (the norm of
    the block's output y, times post_weight) or None. Serves rows of any number and
    float32, float16 or bfloat16."""

    def __init__(self, c, norm="rms", post=None, eps=1e-6, residual_scale=1.0):
        for name, kind in (("norm", norm), ("post", post)):
            if kind is not None and kind not in _NORMS:
                raise ValueError("%s must be one of %s or None" % (name, sorted(_NORMS)))
        if not 1 <= c <= _abi.IS_MAX_NORM_CHANNELS:
            raise ValueError("c must be 1 to %d, got %r" % (_abi.IS_MAX_NORM_CHANNELS, c))
        if not 0 <= eps < float("inf") or (eps > 0 and ctypes.c_float(eps).value == 0.0):
            raise ValueError("eps must be finite, at least 0, and not become 0 in float32, got %r" % (eps,))
        self.c, self.eps, self.residual_scale = c, eps, residual_scale
        self.norm, self.post = _NORMS.get(norm, 0), _NORMS.get(post, 0)
        self._lib, self._layouts = _abi.load(), _Layouts()
        self._current_device, self._current_stream = _device_calls()
        import torch
        self._torch = torch

    def apply(self, x, y=None, gate=None, post_weight=None, weight=None, bias=None, scale=None, shift=None, x_out=None,
              out=None, stream=None):
        """Returns (x_out, out). y None: no block before, x_out is x. x_out and out
        None: new dense tensors; pass x or y to work in place. gate, scale, shift: (n
        or 1) x c of x's dtype; post_weight, weight, bias: c float32 values. stream: a
        hipStream_t in place of torch's current stream; needs the outputs."""
        try:
            key = (_sig(x), _sig(y), _sig(gate), _sig(post_weight), _sig(weight), _sig(bias), _sig(scale), _sig(shift),
                   _sig(x_out), _sig(out))
            call = self._layouts.get(key)
        except AttributeError:      # not a tensor: the checks say so
            key = call = None
        if call is None:
            call = self._layouts.keep(key, self._check_apply(x, y, gate, post_weight, weight, bias, scale, shift, x_out,
                                                             out))
        wants_x, wants_out = y is not None, self.norm != 0
        if stream is not None and ((wants_x and x_out is None) or (wants_out and out is None)):
            raise ValueError("a call on a stream of its own needs x_out and out: %s" % _ALLOCATED)
        if not _one_device((x, y, gate, post_weight, weight, bias, scale, shift, x_out, out)):
            _check_device(x.device, x=x, y=y, gate=gate, post_weight=post_weight, weight=weight, bias=bias, scale=scale,
                          shift=shift, x_out=x_out, out=out)
        index = x.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.apply(x, y, gate, post_weight, weight, bias, scale, shift, x_out, out, stream)
        if wants_x and x_out is None:
            x_out = self._torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if wants_out and out is None:
            out = self._torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.block_norm_forward(call, x.data_ptr() or None, _ptr(y), _ptr(gate), _ptr(post_weight),
                                          _ptr(weight), _ptr(bias), _ptr(scale), _ptr(shift), _ptr(x_out), _ptr(out),
                                          stream or None)
        if st:
            _abi.check(st, "block_norm_forward")
        return (x_out if wants_x else x), out

    def _check_apply(self, x, y, gate, post_weight, weight, bias, scale, shift, x_out, out):
        code = _dtype(x, "x")
        _check_rows(x, "x", x.dtype, self.c)
        if y is not None:
            _check_rows(y, "y", x.dtype, shape=x.shape)
        elif self.post or gate is not None or x_out is not None or post_weight is not None:
            raise ValueError("post, post_weight, gate and x_out need y")
        elif not self.norm:
            raise ValueError("without a norm and y there is nothing to compute")
        if not self.post and post_weight is not None:
            raise ValueError("post_weight needs post")
        if not self.norm and any(t is not None for t in (weight, bias, scale, shift, out)):
            raise ValueError("weight, bias, scale, shift and out need norm")
        strides = [_check_per_entry(t, name, x) for name, t in (("gate", gate), ("scale", scale), ("shift", shift))]
        for name, t in (("post_weight", post_weight), ("weight", weight), ("bias", bias)):
            _check_weight(t, self.c, name)
        for name, t in (("x_out", x_out), ("out", out)):
            if t is not None:
                _check_rows(t, name, x.dtype, shape=x.shape)
        return block_norm_desc(code, self.c, self.norm, self.post, self.eps, self.residual_scale, _rows(x),
                               _rows(x if y is None else y), _rows(x if x_out is None else x_out, x_out is None),
                               _rows(x if out is None else out, out is None), *strides)


def block_norm(x, y=None, norm="rms", post=None, eps=1e-6, residual_scale=1.0, **vectors):
    """(x_out, out) of BlockNorm(x's channels, ...).apply(x, y, **vectors)."""
    return BlockNorm(x.shape[-1], norm, post, eps, residual_scale).apply(x, y, **vectors)


class Dense:
    """The plan of out = residual + act(x w^T + bias) for tensors laid out like x (n x
    len x in), w (features x in), out (n x len x features; None: dense) and residual
    (like out unless given). Only shapes, strides and dtype (float16 or bfloat16) are
    taken from them. activation: "none", "relu", "gelu", "gelu_tanh" or "silu".
    forward() launches on torch's current stream."""

    def __init__(self, x, w, out=None, residual=None, activation="none"):
        import torch
        self._torch = torch
        if activation not in _ACTIVATIONS:
            raise ValueError("activation must be one of %s" % sorted(_ACTIVATIONS))
        code = _dtype(x, "x", f32=False)
        _check_rows(x, "x", x.dtype)
        n, length, k = x.shape
        if not isinstance(w, torch.Tensor) or w.dtype != x.dtype:
            raise TypeError("w must be a %s tensor" % x.dtype)
        if w.dim() != 2 or w.shape[1] != k:
            raise ValueError("w must be features x %d, got shape %s" % (k, tuple(w.shape)))
        if k > 1 and w.stride(1) != 1:
            raise ValueError("w must have a contiguous last dimension")
        m = w.shape[0]
        if m > _INT_MAX:
            raise ValueError("w has a dimension over %d, got shape %s" % (_INT_MAX, tuple(w.shape)))
        shape = torch.Size((n, length, m))
        dense = (length * m, m, 1)
        for name, t in (("out", out), ("residual", residual)):
            if t is not None:
                _check_rows(t, name, x.dtype, shape=shape)
        out_stride = dense if out is None else tuple(out.stride())
        self._like = {"x": (x.shape, x.stride()), "w": (w.shape, w.stride()), "out": (shape, out_stride),
                      "residual": (shape, out_stride if residual is None else tuple(residual.stride()))}
        self.dtype, self.features = x.dtype, m
        S = ctypes.c_int64 * 2
        self._desc = dense_desc(n, length, k, m, code, _ACTIVATIONS[activation],
                                *[S(*self._like[name][1][:2]) for name in ("x", "residual", "out")], w.stride(0))
        self.handle = dense_create(self._desc)
        self._lib, self._layouts = _abi.load(), _Layouts()
        self._current_device, self._current_stream = _device_calls()
        # Bound now: at interpreter exit the module's globals may already be
        # gone when __del__ runs.
        self._destroy = self._lib.dense_destroy
        self.workspace_bytes = dense_workspace_size(self.handle)

    def info(self):
        return dense_get_plan_info(self.handle)

    def new_workspace(self, device="cuda"):
        """A workspace for forward() (None when it needs none). Calls that
        overlap in time, on different streams, need one each."""
        import torch
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device) if self.workspace_bytes else None

    def forward(self, x, w, bias=None, residual=None, out=None, workspace=None, stream=None):
        """Into `out` (None: a new tensor with the strides of the plan's). bias: float32,
        one value a feature; residual: may be `out` itself. workspace: from
        new_workspace() (None: allocated for the call). stream: a hipStream_t in place
        of torch's current stream; needs `out` and the workspace."""
        try:
            key = (_sig(x), _sig(w), _sig(bias), _sig(residual), _sig(out))
            seen = self._layouts.get(key)
        except AttributeError:      # not a tensor: the checks say so
            key = seen = None
        if not seen:
            self._check_forward(x, w, bias, residual, out)
            self._layouts.keep(key, True)
        if workspace is not None:
            if not isinstance(workspace, self._torch.Tensor):
                raise TypeError("workspace must be a tensor")
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        if stream is not None and (out is None or (workspace is None and self.workspace_bytes)):
            raise ValueError("a call on a stream of its own needs out and workspace: %s" % _ALLOCATED)
        if not _one_device((x, w, bias, residual, out, workspace)):
            _check_device(x.device, x=x, w=w, bias=bias, residual=residual, out=out, workspace=workspace)
        index = x.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.forward(x, w, bias, residual, out, workspace, stream)
        if out is None:
            out = self._torch.empty_strided(*self._like["out"], dtype=self.dtype, device=x.device)
        if workspace is None and self.workspace_bytes:
            workspace = self.new_workspace(x.device)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.dense_forward(self.handle, x.data_ptr() or None, w.data_ptr() or None, _ptr(bias),
                                     _ptr(residual), out.data_ptr() or None, _ptr(workspace),
                                     workspace.numel() * workspace.element_size() if workspace is not None else 0,
                                     stream or None)
        if st:
            _abi.check(st, "dense_forward")
        return out

    def _check_forward(self, x, w, bias, residual, out):
        torch = self._torch
        for name, t in (("x", x), ("w", w), ("residual", residual), ("out", out)):
            if t is None and name in ("residual", "out"):
                continue
            shape, stride = self._like[name]
            if not isinstance(t, torch.Tensor) or t.dtype != self.dtype:
                raise TypeError("%s must be a %s tensor" % (name, self.dtype))
            if t.shape != shape or _steps(shape, t.stride()) != _steps(shape, stride):
                raise ValueError("%s is %s with strides %s, the plan is for %s with strides %s"
                                 % (name, tuple(t.shape), t.stride(), tuple(shape), tuple(stride)))
        _check_weight(bias, self.features, "bias")

    def __del__(self):
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h and destroy is not None:
            destroy(h)
            self.handle = None


def dense(x, w, bias=None, activation="none", residual=None):
    """residual + act(x w^T + bias). x: n x len x in, w: features x in (float16 or
    bfloat16); bias: float32; residual: n x len x features."""
    return Dense(x, w, residual=residual, activation=activation).forward(x, w, bias, residual)
