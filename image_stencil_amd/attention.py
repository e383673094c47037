"""Python binding of the attention operators: rotary positions, the norm of
queries and keys with the rotation, and cross attention (include/imgstencil.h).

Tensors are torch device tensors n x len x heads x d with a contiguous last
dimension and any other strides; an fp16 NHWC feature map (n, H, W, C) viewed as
(n, H * W, heads, C // heads) is one. The functions with the C names marshal
arguments to the C ABI and nothing else; Rotary and CrossAttention own a plan,
check their tensors and launch on torch's current stream of the tensors' device.
"""
import ctypes

from . import _abi
from ._abi import cross_attention_desc, conv2d_plan_info, is_tokens, qk_norm_desc, rotary_desc

_LAYOUTS = {"half": _abi.IS_ROTARY_HALF, "interleaved": _abi.IS_ROTARY_INTERLEAVED}
_SCALINGS = {"none": _abi.IS_ROTARY_UNSCALED, "linear": _abi.IS_ROTARY_LINEAR, "ntk": _abi.IS_ROTARY_NTK,
             "ramp": _abi.IS_ROTARY_RAMP}
_NORMS = {"rms": _abi.IS_NORM_RMS, "layer": _abi.IS_NORM_LAYER}
_INT_MAX = 2147483647   # the descriptors hold sizes as int
_ALLOCATED = "memory allocated here belongs to torch's current stream"


# ------------------------------------------------------------------ the C names
def rotary_create(desc):
    """Returns an opaque plan handle (int); raises ImgStencilError on a bad desc."""
    plan = ctypes.c_void_p()
    _abi.check(_abi.load().rotary_create(ctypes.byref(desc), ctypes.byref(plan)), "rotary_create")
    return plan.value


def rotary_destroy(plan):
    _abi.load().rotary_destroy(plan)


def rotary_get_frequencies(plan):
    """The frequencies of one axis after scaling (radians per position)."""
    n = ctypes.c_int()
    arr = (ctypes.c_double * (_abi.IS_MAX_HEAD_DIM // 2))()
    _abi.check(_abi.load().rotary_get_frequencies(plan, arr, len(arr), ctypes.byref(n)), "rotary_get_frequencies")
    return list(arr[:n.value])


def rotary_forward(plan, dtype, xt, x_ptr, pos_ptr, pos_batch_stride, yt, y_ptr, stream):
    """xt, yt: is_tokens; raw pointers (ints) and a hipStream_t (int)."""
    _abi.check(_abi.load().rotary_forward(plan, dtype, xt, x_ptr, pos_ptr or None, pos_batch_stride, yt, y_ptr,
                                          stream or None), "rotary_forward")


def qk_norm_rotary_forward(plan, desc, q_ptr, k_ptr, q_weight_ptr, k_weight_ptr, q_pos_ptr, k_pos_ptr, q_out_ptr,
                           k_out_ptr, stream):
    _abi.check(_abi.load().qk_norm_rotary_forward(plan, ctypes.byref(desc), q_ptr or None, k_ptr or None,
                                                  q_weight_ptr or None, k_weight_ptr or None, q_pos_ptr or None,
                                                  k_pos_ptr or None, q_out_ptr or None, k_out_ptr or None,
                                                  stream or None), "qk_norm_rotary_forward")


def cross_attention_create(desc):
    plan = ctypes.c_void_p()
    _abi.check(_abi.load().cross_attention_create(ctypes.byref(desc), ctypes.byref(plan)), "cross_attention_create")
    return plan.value


def cross_attention_destroy(plan):
    _abi.load().cross_attention_destroy(plan)


def cross_attention_workspace_size(plan):
    n = ctypes.c_size_t()
    _abi.check(_abi.load().cross_attention_workspace_size(plan, ctypes.byref(n)), "cross_attention_workspace_size")
    return n.value


def cross_attention_get_plan_info(plan):
    """grid: (workgroups over all heads and entries, parts of the keys, 1); tile:
    (keys per part, rows of a row tile)."""
    info = conv2d_plan_info()
    _abi.check(_abi.load().cross_attention_get_plan_info(plan, ctypes.byref(info)), "cross_attention_get_plan_info")
    return {"kernel": info.kernel.decode(), "grid": (info.grid_x, info.grid_y, info.grid_z), "block": info.block,
            "lds_bytes": info.lds_bytes, "tile": (info.tile_w, info.tile_h), "flops": info.flops,
            "bytes": info.bytes}


def cross_attention_forward(plan, q_ptr, k_ptr, v_ptr, mask_ptr, lengths_ptr, out_ptr, lse_ptr, ws_ptr, ws_bytes,
                            stream):
    _abi.check(_abi.load().cross_attention_forward(plan, q_ptr or None, k_ptr or None, v_ptr or None, mask_ptr or None,
                                                   lengths_ptr or None, out_ptr or None, lse_ptr or None,
                                                   ws_ptr or None, ws_bytes, stream or None),
               "cross_attention_forward")


# ---------------------------------------------------------------- torch helpers
def _dtype(t, name, f32=True):
    import torch
    known = {torch.float16: _abi.IS_F16, torch.bfloat16: _abi.IS_BF16}
    if f32:
        known[torch.float32] = _abi.IS_F32
    if not isinstance(t, torch.Tensor) or t.dtype not in known:
        raise TypeError("%s must be a %sfloat16 or bfloat16 tensor" % (name, "float32, " if f32 else ""))
    return known[t.dtype]


# Shape, dtype and stride checks come before the device checks, so that every
# rejected argument is reported the same way with or without a GPU.
def _check_tokens(t, name, dtype, d=None):
    import torch
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError("%s must be a %s tensor" % (name, dtype))
    if t.dim() != 4:
        raise ValueError("%s must be n x len x heads x d, got shape %s" % (name, tuple(t.shape)))
    if max(t.shape) > _INT_MAX:
        raise ValueError("%s has a dimension over %d, got shape %s" % (name, _INT_MAX, tuple(t.shape)))
    if d is not None and t.shape[3] != d:
        raise ValueError("%s has %d elements per head, expected %d" % (name, t.shape[3], d))
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)


def _check_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != device):
            raise TypeError("%s must be a tensor on %s" % (name, device if device.type == "cuda" else "a GPU"))


def _tokens(t, dense=False):
    """The token tensor t, or a new dense one of its shape."""
    n, length, heads, d = t.shape
    s = (length * heads * d, heads * d, d) if dense else t.stride()
    return is_tokens(n, length, heads, s[0], s[1], s[2])


def _check_positions(pos, t, axes, name):
    """int32, (n or 1) x len x axes, or (n or 1) x len for one axis; returns the
    batch stride in elements (0: one row set for the whole batch)."""
    import torch
    if not isinstance(pos, torch.Tensor) or pos.dtype != torch.int32:
        raise TypeError("%s must be an int32 tensor" % name)
    shape = tuple(pos.shape) + ((1,) if pos.dim() == 2 and axes == 1 else ())
    if len(shape) != 3 or shape[0] not in (1, t.shape[0]) or shape[1] != t.shape[1] or shape[2] != axes:
        raise ValueError("%s must be %d (or 1) x %d x %d, got shape %s" % (name, t.shape[0], t.shape[1], axes,
                                                                          tuple(pos.shape)))
    if not pos[:1].is_contiguous():
        raise ValueError("%s must have contiguous rows" % name)
    return 0 if shape[0] == 1 else pos.stride(0)


def _check_weight(w, d, name):
    import torch
    if w is None:
        return
    if not isinstance(w, torch.Tensor) or w.dtype != torch.float32:
        raise TypeError("%s must be a float32 tensor" % name)
    if tuple(w.shape) != (d,) or not w.is_contiguous():
        raise ValueError("%s must hold %d contiguous values, got shape %s" % (name, d, tuple(w.shape)))


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _sig(t):
    """What a layout check looks at."""
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _device_calls():
    """(the current device's index, the current stream of a device as a number).
    torch's raw forms, bound once per plan: building a Stream object costs a
    microsecond, a quarter of a small call."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
            raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream)


def _one_device(tensors):
    """True when all tensors that are given lie on one GPU."""
    d = tensors[0].get_device()
    if d < 0 or not tensors[0].is_cuda:
        return False
    for t in tensors:
        if t is not None and (t.get_device() != d or not t.is_cuda):
            return False
    return True


class _Layouts(dict):
    """Checked layouts of a plan's calls: shapes, strides and dtypes (never
    addresses) -> the C arguments that follow from them. A call with a layout
    seen before skips its checks. Few layouts recur in a program; a stray
    thousand starts over."""
    LIMIT = 256

    def keep(self, key, value):
        if len(self) >= self.LIMIT:
            self.clear()
        self[key] = value
        return value


class Rotary:
    """Rotary positions for heads of d elements, the first `rot` of which turn
    (None: all). axes: positions per token (2: row and column of an image);
    layout "half" or "interleaved"; scaling "none", "linear", "ntk" or "ramp"
    (see rotary_desc in include/imgstencil.h): factor, and for "ramp" the trained
    length original_len and ramp = (low, high) in turns over it; magnitude
    multiplies what turns. Serves tensors of any length, dtype and head count."""

    def __init__(self, d, rot=None, axes=1, layout="half", base=10000.0, scaling="none", factor=1.0,
                 original_len=0, ramp=(1.0, 32.0), magnitude=1.0):
        if layout not in _LAYOUTS:
            raise ValueError("layout must be one of %s" % sorted(_LAYOUTS))
        if scaling not in _SCALINGS:
            raise ValueError("scaling must be one of %s" % sorted(_SCALINGS))
        self.d, self.rot, self.axes = d, d if rot is None else rot, axes
        desc = rotary_desc(d, self.rot, axes, _LAYOUTS[layout], _SCALINGS[scaling], original_len, base, factor,
                           ramp[0], ramp[1], magnitude)
        self.handle = rotary_create(desc)
        self._lib, self._layouts = _abi.load(), _Layouts()
        self._current_device, self._current_stream = _device_calls()
        # Bound now: at interpreter exit the module's globals may already be
        # gone when __del__ runs.
        self._destroy = self._lib.rotary_destroy
        import torch
        self._torch = torch

    def frequencies(self):
        return rotary_get_frequencies(self.handle)

    def apply(self, x, positions, out=None, stream=None):
        """x rotated, into `out` (x itself: in place; None: a new dense tensor).
        positions: int32, (n or 1) x len x axes. stream: a hipStream_t in place
        of torch's current stream; needs `out`."""
        try:
            key = (x.shape, x.stride(), x.dtype, positions.shape, positions.stride(), positions.dtype, _sig(out))
            call = self._layouts.get(key)
        except AttributeError:      # not a tensor: the checks say so
            key = call = None
        if call is None:
            call = self._layouts.keep(key, self._check_apply(x, positions, out))
        if stream is not None and out is None:
            raise ValueError("a call on a stream of its own needs out: %s" % _ALLOCATED)
        if not _one_device((x, positions, out)):
            _check_device(x.device, x=x, positions=positions, out=out)
        index = x.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.apply(x, positions, out, stream)
        if out is None:
            out = self._torch.empty(x.shape, dtype=x.dtype, device=x.device)
        code, xt, pb, yt = call
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.rotary_forward(self.handle, code, xt, x.data_ptr(), positions.data_ptr() or None, pb, yt,
                                      out.data_ptr(), stream or None)
        if st:
            _abi.check(st, "rotary_forward")
        return out

    def _check_apply(self, x, positions, out):
        code = _dtype(x, "x")
        _check_tokens(x, "x", x.dtype, self.d)
        pb = _check_positions(positions, x, self.axes, "positions")
        if out is not None:
            _check_tokens(out, "out", x.dtype, self.d)
            if out.shape != x.shape:
                raise ValueError("out has shape %s, x %s" % (tuple(out.shape), tuple(x.shape)))
        return code, _tokens(x), pb, _tokens(x if out is None else out, out is None)

    def apply_qk_norm(self, q, k, q_positions, k_positions=None, q_weight=None, k_weight=None, eps=1e-6,
                      norm="rms", q_out=None, k_out=None, stream=None):
        """The norm ("rms" or "layer") of every head of q and k, times the fp32
        weights (None: ones), rotated. k_positions None: those of q. Returns
        (q_out, k_out); pass q and k themselves to work in place. stream: as in
        apply; needs both outputs."""
        if k_positions is None:
            k_positions = q_positions
        try:
            key = (_sig(q), _sig(k), _sig(q_positions), _sig(k_positions), _sig(q_weight), _sig(k_weight), eps, norm,
                   _sig(q_out), _sig(k_out))
            call = self._layouts.get(key)
        except (AttributeError, TypeError):     # not a tensor, no number: the checks say so
            key = call = None
        if call is None:
            call = self._layouts.keep(key, self._check_qk_norm(q, k, q_positions, k_positions, q_weight, k_weight, eps,
                                                               norm, q_out, k_out))
        if stream is not None and (q_out is None or k_out is None):
            raise ValueError("a call on a stream of its own needs q_out and k_out: %s" % _ALLOCATED)
        if not _one_device((q, k, q_positions, k_positions, q_weight, k_weight, q_out, k_out)):
            _check_device(q.device, q=q, k=k, q_positions=q_positions, k_positions=k_positions, q_weight=q_weight,
                          k_weight=k_weight, q_out=q_out, k_out=k_out)
        index = q.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.apply_qk_norm(q, k, q_positions, k_positions, q_weight, k_weight, eps, norm, q_out, k_out,
                                          stream)
        if q_out is None:
            q_out = self._torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_out is None:
            k_out = self._torch.empty(k.shape, dtype=k.dtype, device=k.device)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.qk_norm_rotary_forward(self.handle, call, q.data_ptr() or None, k.data_ptr() or None,
                                              _ptr(q_weight), _ptr(k_weight), q_positions.data_ptr() or None,
                                              k_positions.data_ptr() or None, q_out.data_ptr() or None,
                                              k_out.data_ptr() or None, stream or None)
        if st:
            _abi.check(st, "qk_norm_rotary_forward")
        return q_out, k_out

    def _check_qk_norm(self, q, k, q_positions, k_positions, q_weight, k_weight, eps, norm, q_out, k_out):
        code = _dtype(q, "q")
        _check_tokens(q, "q", q.dtype, self.d)
        _check_tokens(k, "k", q.dtype, self.d)
        if eps > 0 and ctypes.c_float(eps).value == 0.0:
            raise ValueError("eps must not become 0 in float32, got %r" % (eps,))
        if norm not in _NORMS:
            raise ValueError("norm must be one of %s" % sorted(_NORMS))
        qb = _check_positions(q_positions, q, self.axes, "q_positions")
        kb = _check_positions(k_positions, k, self.axes, "k_positions")
        _check_weight(q_weight, self.d, "q_weight")
        _check_weight(k_weight, self.d, "k_weight")
        for name, o, t in (("q_out", q_out, q), ("k_out", k_out, k)):
            if o is not None:
                _check_tokens(o, name, q.dtype, self.d)
                if o.shape != t.shape:
                    raise ValueError("%s has shape %s, expected %s" % (name, tuple(o.shape), tuple(t.shape)))
        return qk_norm_desc(code, _NORMS[norm], eps, _tokens(q), _tokens(k), _tokens(q if q_out is None else q_out,
                            q_out is None), _tokens(k if k_out is None else k_out, k_out is None), qb, kb)

    def __del__(self):
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h and destroy is not None:
            destroy(h)
            self.handle = None


def _check_qkv(q, k, v):
    _check_tokens(q, "q", q.dtype)
    _check_tokens(k, "k", q.dtype, q.shape[3])
    _check_tokens(v, "v", q.dtype, q.shape[3])
    if v.shape != k.shape:
        raise ValueError("k has shape %s, v %s" % (tuple(k.shape), tuple(v.shape)))
    if k.shape[0] != q.shape[0]:
        raise ValueError("q has %d batch entries, k and v %d" % (q.shape[0], k.shape[0]))
    if k.shape[2] == 0 or q.shape[2] % k.shape[2]:
        raise ValueError("%d query heads do not share %d key heads evenly" % (q.shape[2], k.shape[2]))


def _steps(shape, stride):
    """The strides that lead from one element to another: not those of dimensions
    of one element, and none of an empty tensor's."""
    return None if 0 in shape else tuple(s if n > 1 else 0 for n, s in zip(shape, stride))


class CrossAttention:
    """The plan of cross attention for tensors laid out like q (n x lq x hq x d),
    k and v (n x lk x hkv x d) and out (like q; None: dense). Only shapes,
    strides and dtype are taken from them. scale None: 1 / sqrt(d).
    forward() launches on torch's current stream."""

    def __init__(self, q, k, v, out=None, scale=None):
        import torch
        self._torch = torch
        code = _dtype(q, "q", f32=False)
        _check_qkv(q, k, v)
        if out is not None:
            _check_tokens(out, "out", q.dtype, q.shape[3])
            if out.shape != q.shape:
                raise ValueError("out has shape %s, q %s" % (tuple(out.shape), tuple(q.shape)))
        # Held in fp32, where 0 stands for 1 / sqrt(d).
        if scale is not None and ctypes.c_float(scale).value == 0.0:
            raise ValueError("scale must not be 0 in float32, got %r" % (scale,))
        n, lq, hq, d = q.shape
        lk, hkv = k.shape[1], k.shape[2]
        dense = (lq * hq * d, hq * d, d, 1)
        self._like = tuple((tuple(t.shape), tuple(t.stride())) for t in (q, k, v)) + (
            (tuple(q.shape), dense if out is None else tuple(out.stride())),)
        self.dtype = q.dtype
        S = ctypes.c_int64 * 3
        self._desc = cross_attention_desc(n, lq, lk, hq, hkv, d, code, 0.0 if scale is None else scale,
                                          *[S(*st[:3]) for (_, st) in self._like], lk)
        self.handle = cross_attention_create(self._desc)
        self._lib, self._layouts = _abi.load(), _Layouts()
        self._current_device, self._current_stream = _device_calls()
        self._destroy = self._lib.cross_attention_destroy
        self.workspace_bytes = cross_attention_workspace_size(self.handle)

    def info(self):
        return cross_attention_get_plan_info(self.handle)

    def new_workspace(self, device="cuda"):
        """A workspace for forward() (None when it needs none). Calls that
        overlap in time, on different streams, need one each."""
        import torch
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device) if self.workspace_bytes else None

    def forward(self, q, k, v, out=None, key_mask=None, key_lengths=None, lse=None, workspace=None, stream=None):
        """Attention into `out` (None: a new tensor with the strides of the plan's,
        dense unless the plan was made for another). key_mask: bool or uint8,
        n x lk, true where a key is visible; key_lengths: int32, n; lse: float32,
        n x hq x lq, receives the log-sum-exp of each row. workspace: from
        new_workspace() (None: allocated for the call)."""
        try:
            key = (_sig(q), _sig(k), _sig(v), _sig(out), _sig(key_mask), _sig(key_lengths), _sig(lse))
            seen = self._layouts.get(key)
        except AttributeError:      # not a tensor: the checks say so
            key = seen = None
        if not seen:
            self._check_forward(q, k, v, out, key_mask, key_lengths, lse)
            self._layouts.keep(key, True)
        if workspace is not None:
            if not isinstance(workspace, self._torch.Tensor):
                raise TypeError("workspace must be a tensor")
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        if stream is not None and (out is None or (workspace is None and self.workspace_bytes)):
            raise ValueError("a call on a stream of its own needs out and workspace: %s" % _ALLOCATED)
        if not _one_device((q, k, v, out, key_mask, key_lengths, lse, workspace)):
            _check_device(q.device, q=q, k=k, v=v, out=out, key_mask=key_mask, key_lengths=key_lengths, lse=lse,
                          workspace=workspace)
        index = q.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.forward(q, k, v, out, key_mask, key_lengths, lse, workspace, stream)
        if out is None:
            out = self._torch.empty_strided(*self._like[3], dtype=self.dtype, device=q.device)
        if workspace is None and self.workspace_bytes:
            workspace = self.new_workspace(q.device)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.cross_attention_forward(self.handle, q.data_ptr() or None, k.data_ptr() or None,
                                               v.data_ptr() or None, _ptr(key_mask), _ptr(key_lengths),
                                               out.data_ptr() or None, _ptr(lse), _ptr(workspace),
                                               workspace.numel() * workspace.element_size()
                                               if workspace is not None else 0, stream or None)
        if st:
            _abi.check(st, "cross_attention_forward")
        return out

    def _check_forward(self, q, k, v, out, key_mask, key_lengths, lse):
        torch = self._torch
        for name, t, (shape, stride) in zip(("q", "k", "v", "out"), (q, k, v, out), self._like):
            if t is None and name == "out":
                continue
            if not isinstance(t, torch.Tensor) or t.dtype != self.dtype:
                raise TypeError("%s must be a %s tensor" % (name, self.dtype))
            if t.shape != shape or _steps(shape, t.stride()) != _steps(shape, stride):
                raise ValueError("%s is %s with strides %s, the plan is for %s with strides %s"
                                 % (name, tuple(t.shape), t.stride(), shape, stride))
        n, lq, hq, lk = self._desc.n, self._desc.lq, self._desc.hq, self._desc.lk
        if key_mask is not None:
            if not isinstance(key_mask, torch.Tensor) or key_mask.dtype not in (torch.bool, torch.uint8):
                raise TypeError("key_mask must be a bool or uint8 tensor")
            if key_mask.shape != (n, lk) or not key_mask.is_contiguous():
                raise ValueError("key_mask must be a contiguous %d x %d, got shape %s" % (n, lk, tuple(key_mask.shape)))
        if key_lengths is not None:
            if not isinstance(key_lengths, torch.Tensor) or key_lengths.dtype != torch.int32:
                raise TypeError("key_lengths must be an int32 tensor")
            if key_lengths.shape != (n,) or not key_lengths.is_contiguous():
                raise ValueError("key_lengths must hold %d values, got shape %s" % (n, tuple(key_lengths.shape)))
        if lse is not None:
            if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32:
                raise TypeError("lse must be a float32 tensor")
            if lse.shape != (n, hq, lq) or not lse.is_contiguous():
                raise ValueError("lse must be a contiguous %d x %d x %d, got shape %s" % (n, hq, lq, tuple(lse.shape)))

    def __del__(self):
        h = getattr(self, "handle", None)
        destroy = getattr(self, "_destroy", None)
        if h and destroy is not None:
            destroy(h)
            self.handle = None


def rotary(x, positions, plan, out=None):
    """x rotated by the Rotary `plan` (see Rotary.apply)."""
    return plan.apply(x, positions, out=out)


def qk_norm_rotary(q, k, q_positions, plan, k_positions=None, q_weight=None, k_weight=None, eps=1e-6, norm="rms"):
    """Normed and rotated queries and keys (see Rotary.apply_qk_norm)."""
    return plan.apply_qk_norm(q, k, q_positions, k_positions, q_weight, k_weight, eps, norm)


def cross_attention(q, k, v, key_mask=None, key_lengths=None, scale=None, return_lse=False):
    """softmax(scale * q k^T) v over the visible keys. q: n x lq x hq x d; k, v:
    n x lk x hkv x d (fp16 or bf16). With return_lse also the n x hq x lq fp32
    log-sum-exp of the rows."""
    import torch
    plan = CrossAttention(q, k, v, scale=scale)
    lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device) \
        if return_lse else None
    out = plan.forward(q, k, v, key_mask=key_mask, key_lengths=key_lengths, lse=lse)
    return (out, lse) if return_lse else out
