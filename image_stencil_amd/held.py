"""Python binding of states held in 8 bits and of the cross attention to them
(include/imgstencil.h).

HeldStates keeps the keys and values that are attended to many times (a reference's,
a prompt's) as e4m3 numbers with a power of two for each block of 32 tokens and head;
HeldAttention is CrossAttention with a HeldStates in the place of k and v. The
functions with the C names marshal arguments to the C ABI and nothing else; the
classes check their tensors and launch on torch's current stream of the tensors' device.
"""
import ctypes

from . import _abi
from ._abi import conv2d_plan_info, held_attention_desc, held_states_desc
from .attention import (_ALLOCATED, _INT_MAX, _Layouts, _check_device, _check_tokens, _device_calls, _dtype, _one_device,
                        _ptr, _sig, _steps, _tokens)


# ------------------------------------------------------------------ the C names
def held_states_size(desc):
    n = ctypes.c_size_t()
    _abi.check(_abi.load().held_states_size(ctypes.byref(desc), ctypes.byref(n)), "held_states_size")
    return n.value


def held_store(desc, kt, k_ptr, vt, v_ptr, mask_ptr, mask_stride, lengths_ptr, at, held_ptr, held_bytes, stream):
    """kt, vt: is_tokens; raw pointers (ints) and a hipStream_t (int)."""
    _abi.check(_abi.load().held_store(ctypes.byref(desc), ctypes.byref(kt), k_ptr or None, ctypes.byref(vt),
                                      v_ptr or None, mask_ptr or None, mask_stride, lengths_ptr or None, at,
                                      held_ptr or None, held_bytes, stream or None), "held_store")


def held_load(desc, held_ptr, held_bytes, at, kt, k_ptr, vt, v_ptr, stream):
    _abi.check(_abi.load().held_load(ctypes.byref(desc), held_ptr or None, held_bytes, at, ctypes.byref(kt),
                                     k_ptr or None, ctypes.byref(vt), v_ptr or None, stream or None), "held_load")


def held_attention_create(desc):
    """Returns an opaque plan handle (int); raises ImgStencilError on a bad desc."""
    plan = ctypes.c_void_p()
    _abi.check(_abi.load().held_attention_create(ctypes.byref(desc), ctypes.byref(plan)), "held_attention_create")
    return plan.value


def held_attention_destroy(plan):
    _abi.load().held_attention_destroy(plan)


def held_attention_workspace_size(plan):
    n = ctypes.c_size_t()
    _abi.check(_abi.load().held_attention_workspace_size(plan, ctypes.byref(n)), "held_attention_workspace_size")
    return n.value


def held_attention_get_plan_info(plan):
    """grid: (workgroups over all heads and entries, parts of the keys, 1); tile:
    (keys per part, rows of a row tile)."""
    info = conv2d_plan_info()
    _abi.check(_abi.load().held_attention_get_plan_info(plan, ctypes.byref(info)), "held_attention_get_plan_info")
    return {"kernel": info.kernel.decode(), "grid": (info.grid_x, info.grid_y, info.grid_z), "block": info.block,
            "lds_bytes": info.lds_bytes, "tile": (info.tile_w, info.tile_h), "flops": info.flops, "bytes": info.bytes}


def held_attention_forward(plan, q_ptr, held_ptr, held_bytes, mask_ptr, lengths_ptr, out_ptr, lse_ptr, ws_ptr, ws_bytes,
                           stream):
    _abi.check(_abi.load().held_attention_forward(plan, q_ptr or None, held_ptr or None, held_bytes, mask_ptr or None,
                                                  lengths_ptr or None, out_ptr or None, lse_ptr or None, ws_ptr or None,
                                                  ws_bytes, stream or None), "held_attention_forward")


# ---------------------------------------------------------------- torch helpers
def _check_keys(n, length, key_mask, key_lengths):
    import torch
    if key_mask is not None:
        if not isinstance(key_mask, torch.Tensor) or key_mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("key_mask must be a bool or uint8 tensor")
        if key_mask.shape != (n, length) or not key_mask.is_contiguous():
            raise ValueError("key_mask must be a contiguous %d x %d, got shape %s" % (n, length, tuple(key_mask.shape)))
    if key_lengths is not None:
        if not isinstance(key_lengths, torch.Tensor) or key_lengths.dtype != torch.int32:
            raise TypeError("key_lengths must be an int32 tensor")
        if key_lengths.shape != (n,) or not key_lengths.is_contiguous():
            raise ValueError("key_lengths must hold %d values, got shape %s" % (n, tuple(key_lengths.shape)))


class HeldStates:
    """Keys and values of n entries, up to `length` tokens and `heads` key heads of d
    elements (a multiple of 8), held in 8 bits on `device`; zeros at first. dtype
    (float16 or bfloat16) is that of the tensors put in and got out and of the queries.
    The constructor waits until the zeros are there, so that any stream may use the
    store; made while torch's current stream is captured, it is cleared by the graph."""

    def __init__(self, n, length, heads, d, dtype=None, device="cuda"):
        import torch
        self._torch = torch
        codes = {torch.float16: _abi.IS_F16, torch.bfloat16: _abi.IS_BF16}
        dtype = torch.float16 if dtype is None else dtype
        if dtype not in codes:
            raise TypeError("dtype must be float16 or bfloat16, got %s" % (dtype,))
        if max(n, length, heads, d) > _INT_MAX:
            raise ValueError("sizes must be at most %d" % _INT_MAX)
        self.n, self.length, self.heads, self.d, self.dtype = n, length, heads, d, dtype
        self.desc = held_states_desc(n, length, heads, d, codes[dtype])
        self.bytes = held_states_size(self.desc)
        self.data = torch.zeros(self.bytes, dtype=torch.uint8, device=device)
        if self.data.is_cuda:
            with torch.cuda.device(self.data.get_device()):
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().synchronize()
        self._ref = ctypes.byref(self.desc)
        self._lib, self._layouts = _abi.load(), _Layouts()
        self._current_device, self._current_stream = _device_calls()

    def put(self, k, v, at=0, key_mask=None, key_lengths=None, stream=None):
        """k and v (n x len x heads x d) become tokens at .. at + len - 1 of every entry;
        `at` is a multiple of 32, and a last block that they only begin is filled with
        zeros. Tokens beyond key_lengths (int32, n) or where key_mask (bool or uint8, n
        x len) is false are held as zeros, whatever k and v have there. stream: a
        hipStream_t in place of torch's current stream."""
        try:
            key = (_sig(k), _sig(v), at, _sig(key_mask), _sig(key_lengths))
            call = self._layouts.get(key)
        except (AttributeError, TypeError):      # not a tensor, no number: the checks say so
            key = call = None
        if call is None:
            self._check_sides(k, v, at, "k", "v")
            if at % _abi.IS_HELD_BLOCK:
                raise ValueError("at must be a multiple of %d, got %r" % (_abi.IS_HELD_BLOCK, at))
            _check_keys(self.n, k.shape[1], key_mask, key_lengths)
            kt, vt = _tokens(k), _tokens(v)
            call = self._layouts.keep(key, (kt, vt, ctypes.byref(kt), ctypes.byref(vt), k.shape[1]))
        if not _one_device((self.data, k, v, key_mask, key_lengths)):
            _check_device(self.data.device, held=self.data, k=k, v=v, key_mask=key_mask, key_lengths=key_lengths)
        index = self.data.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.put(k, v, at, key_mask, key_lengths, stream)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.held_store(self._ref, call[2], k.data_ptr() or None, call[3], v.data_ptr() or None,
                                  _ptr(key_mask), call[4], _ptr(key_lengths), at, self.data.data_ptr() or None, self.bytes,
                                  stream or None)
        if st:
            _abi.check(st, "held_store")
        return self

    def get(self, at=0, length=None, k_out=None, v_out=None, stream=None):
        """(k, v) of tokens at .. at + length - 1 (None: to the end), into k_out and v_out
        (None: new dense tensors). stream: as in put; needs the outputs."""
        try:
            key = (at, length, _sig(k_out), _sig(v_out))
            call = self._layouts.get(key)
        except (AttributeError, TypeError):
            key = call = None
        if call is None:
            call = self._layouts.keep(key, self._check_get(at, length, k_out, v_out))
        kt, vt, shape = call
        if stream is not None and (k_out is None or v_out is None):
            raise ValueError("a call on a stream of its own needs k_out and v_out: %s" % _ALLOCATED)
        if not _one_device((self.data, k_out, v_out)):
            _check_device(self.data.device, held=self.data, k_out=k_out, v_out=v_out)
        index = self.data.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.get(at, length, k_out, v_out, stream)
        if k_out is None:
            k_out = self._torch.empty(shape, dtype=self.dtype, device=self.data.device)
        if v_out is None:
            v_out = self._torch.empty(shape, dtype=self.dtype, device=self.data.device)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.held_load(self._ref, self.data.data_ptr() or None, self.bytes, at, kt, k_out.data_ptr() or None, vt,
                                 v_out.data_ptr() or None, stream or None)
        if st:
            _abi.check(st, "held_load")
        return k_out, v_out

    def _check_get(self, at, length, k_out, v_out):
        length = self.length - at if length is None else length
        if at < 0 or length < 0 or at + length > self.length:
            raise ValueError("tokens %r to %r of %d" % (at, at + length, self.length))
        like = self._torch.empty((self.n, length, self.heads, self.d), dtype=self.dtype, device="meta")
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None:
                _check_tokens(t, name, self.dtype, self.d)
                if t.shape != like.shape:
                    raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(like.shape)))
        return _tokens(like if k_out is None else k_out), _tokens(like if v_out is None else v_out), like.shape

    def _check_sides(self, k, v, at, *names):
        for name, t in zip(names, (k, v)):
            _check_tokens(t, name, self.dtype, self.d)
            if t.shape[0] != self.n or t.shape[2] != self.heads:
                raise ValueError("%s must be %d x len x %d x %d, got shape %s" % (name, self.n, self.heads, self.d,
                                                                                 tuple(t.shape)))
        if k.shape != v.shape:
            raise ValueError("k has shape %s, v %s" % (tuple(k.shape), tuple(v.shape)))
        if at < 0 or at + k.shape[1] > self.length:
            raise ValueError("tokens %r to %r of %d" % (at, at + k.shape[1], self.length))


class HeldAttention:
    """The plan of cross attention for queries laid out like q (n x lq x hq x d), states
    held like `held` and out (like q; None: dense). Only shapes, strides and dtype are
    taken from them. scale None: 1 / sqrt(d). forward() launches on torch's current
    stream."""

    def __init__(self, q, held, out=None, scale=None):
        import torch
        self._torch = torch
        if not isinstance(held, HeldStates):
            raise TypeError("held must be a HeldStates")
        _dtype(q, "q", f32=False)
        _check_tokens(q, "q", held.dtype, held.d)
        n, lq, hq, d = q.shape
        if n != held.n:
            raise ValueError("q has %d batch entries, the held states %d" % (n, held.n))
        if hq == 0 or hq % held.heads:
            raise ValueError("%d query heads do not share %d key heads evenly" % (hq, held.heads))
        if out is not None:
            _check_tokens(out, "out", q.dtype, d)
            if out.shape != q.shape:
                raise ValueError("out has shape %s, q %s" % (tuple(out.shape), tuple(q.shape)))
        # Held in fp32, where 0 stands for 1 / sqrt(d).
        if scale is not None and ctypes.c_float(scale).value == 0.0:
            raise ValueError("scale must not be 0 in float32, got %r" % (scale,))
        dense = (lq * hq * d, hq * d, d, 1)
        self._like = ((tuple(q.shape), tuple(q.stride())), (tuple(q.shape), dense if out is None else tuple(out.stride())))
        self.dtype, self._held = q.dtype, (held.n, held.length, held.heads, held.d, held.dtype)
        S = ctypes.c_int64 * 3
        self._desc = held_attention_desc(held.desc, lq, hq, 0.0 if scale is None else scale,
                                         *[S(*st[:3]) for (_, st) in self._like], held.length)
        self.handle = held_attention_create(self._desc)
        self._lib, self._layouts = _abi.load(), _Layouts()
        self._current_device, self._current_stream = _device_calls()
        self._destroy = self._lib.held_attention_destroy
        self.workspace_bytes = held_attention_workspace_size(self.handle)

    def info(self):
        return held_attention_get_plan_info(self.handle)

    def new_workspace(self, device="cuda"):
        """A workspace for forward() (None when it needs none). Calls that
        overlap in time, on different streams, need one each."""
        import torch
        return torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device) if self.workspace_bytes else None

    def forward(self, q, held, out=None, key_mask=None, key_lengths=None, lse=None, workspace=None, stream=None):
        """Attention into `out` (None: a new tensor with the strides of the plan's).
        key_mask: bool or uint8, n x held.length, true where a key is visible;
        key_lengths: int32, n; lse: float32, n x hq x lq, receives the log-sum-exp of
        each row. workspace: from new_workspace() (None: allocated for the call)."""
        try:
            key = (_sig(q), held.n, held.length, held.heads, held.d, held.dtype, _sig(out), _sig(key_mask),
                   _sig(key_lengths), _sig(lse))
            seen = self._layouts.get(key)
            data, size = held.data, held.bytes
        except AttributeError:      # not a tensor, no states: the checks say so
            key = seen = None
        if not seen:
            self._check_forward(q, held, out, key_mask, key_lengths, lse)
            self._layouts.keep(key, True)
            data, size = held.data, held.bytes
        if workspace is not None:
            if not isinstance(workspace, self._torch.Tensor):
                raise TypeError("workspace must be a tensor")
            if not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous")
        if stream is not None and (out is None or (workspace is None and self.workspace_bytes)):
            raise ValueError("a call on a stream of its own needs out and workspace: %s" % _ALLOCATED)
        if not _one_device((q, data, out, key_mask, key_lengths, lse, workspace)):
            _check_device(q.device, q=q, held=data, out=out, key_mask=key_mask, key_lengths=key_lengths, lse=lse,
                          workspace=workspace)
        index = q.get_device()
        if self._current_device() != index:     # a launch goes to the current device
            with self._torch.cuda.device(index):
                return self.forward(q, held, out, key_mask, key_lengths, lse, workspace, stream)
        if out is None:
            out = self._torch.empty_strided(*self._like[1], dtype=self.dtype, device=q.device)
        if workspace is None and self.workspace_bytes:
            workspace = self.new_workspace(q.device)
        if stream is None:
            stream = self._current_stream(index)
        st = self._lib.held_attention_forward(self.handle, q.data_ptr() or None, data.data_ptr() or None, size,
                                              _ptr(key_mask), _ptr(key_lengths), out.data_ptr() or None, _ptr(lse),
                                              _ptr(workspace), workspace.numel() * workspace.element_size()
                                              if workspace is not None else 0, stream or None)
        if st:
            _abi.check(st, "held_attention_forward")
        return out

    def _check_forward(self, q, held, out, key_mask, key_lengths, lse):
        torch = self._torch
        if not isinstance(held, HeldStates):
            raise TypeError("held must be a HeldStates")
        if (held.n, held.length, held.heads, held.d, held.dtype) != self._held:
            raise ValueError("held has (n, length, heads, d, dtype) %s, the plan is for %s"
                             % ((held.n, held.length, held.heads, held.d, held.dtype), self._held))
        for name, t, (shape, stride) in zip(("q", "out"), (q, out), self._like):
            if t is None and name == "out":
                continue
            if not isinstance(t, torch.Tensor) or t.dtype != self.dtype:
                raise TypeError("%s must be a %s tensor" % (name, self.dtype))
            if t.shape != shape or _steps(shape, t.stride()) != _steps(shape, stride):
                raise ValueError("%s is %s with strides %s, the plan is for %s with strides %s"
                                 % (name, tuple(t.shape), t.stride(), shape, stride))
        n, (_, lq, hq, _) = held.n, self._like[0][0]
        _check_keys(n, held.length, key_mask, key_lengths)
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


def held_attention(q, held, key_mask=None, key_lengths=None, scale=None, return_lse=False):
    """softmax(scale * q k^T) v over the visible keys of a HeldStates. q: n x lq x hq x
    d. With return_lse also the n x hq x lq fp32 log-sum-exp of the rows."""
    import torch
    plan = HeldAttention(q, held, scale=scale)
    lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device) \
        if return_lse else None
    out = plan.forward(q, held, key_mask=key_mask, key_lengths=key_lengths, lse=lse)
    return (out, lse) if return_lse else out
