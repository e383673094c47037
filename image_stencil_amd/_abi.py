"""ctypes declarations of include/imgstencil.h (argument marshalling only).

Every computation happens in libimgstencil.so (HIP kernels for gfx950). If the
library is not built, loading fails loudly: there is no other code path.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libimgstencil.so")

IS_OK, IS_ERR_INVALID_ARG, IS_ERR_UNSUPPORTED, IS_ERR_MISALIGNED, IS_ERR_HIP, IS_ERR_NO_MEMORY, \
    IS_ERR_WORKSPACE = range(7)
IS_F32, IS_F16, IS_BF16 = 0, 1, 2
IS_NCHW, IS_NHWC = 0, 1
IS_CHAIN_AUTO, IS_CHAIN_FUSED, IS_CHAIN_UNFUSED = 0, 1, 2
IS_ROTARY_HALF, IS_ROTARY_INTERLEAVED = 0, 1
IS_ROTARY_UNSCALED, IS_ROTARY_LINEAR, IS_ROTARY_NTK, IS_ROTARY_RAMP = 0, 1, 2, 3
IS_NORM_RMS, IS_NORM_LAYER = 1, 2
IS_MAX_HEAD_DIM = 256
IS_MAX_NORM_CHANNELS = 16384
IS_ACT_NONE, IS_ACT_RELU, IS_ACT_GELU, IS_ACT_GELU_TANH, IS_ACT_SILU = 0, 1, 2, 3, 4
IS_HELD_BLOCK = 32
IS_MAX_CHAIN = 8
IS_NOALLOC_MAX_WORKSPACE = 256 << 20

STATUS_NAMES = {0: "IS_OK", 1: "IS_ERR_INVALID_ARG", 2: "IS_ERR_UNSUPPORTED", 3: "IS_ERR_MISALIGNED",
                4: "IS_ERR_HIP", 5: "IS_ERR_NO_MEMORY", 6: "IS_ERR_WORKSPACE"}


class conv2d_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in
                ("n", "c", "h", "w", "k", "r", "s", "pad_h", "pad_w", "stride_h", "stride_w",
                 "in_dtype", "out_dtype", "layout", "relu", "separable")]


class conv2d_plan_info(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char * 64), ("grid_x", ctypes.c_int), ("grid_y", ctypes.c_int),
                ("grid_z", ctypes.c_int), ("block", ctypes.c_int), ("lds_bytes", ctypes.c_int),
                ("tile_w", ctypes.c_int), ("tile_h", ctypes.c_int), ("flops", ctypes.c_double),
                ("bytes", ctypes.c_double)]


class conv2d_variant(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char * 64), ("param", ctypes.c_int), ("is_default", ctypes.c_int),
                ("ms", ctypes.c_float)]


class conv_layer_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("c", "k", "r", "s", "relu")]


class conv_chain_desc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("h", ctypes.c_int), ("w", ctypes.c_int), ("n_layers", ctypes.c_int),
                ("layer", conv_layer_desc * IS_MAX_CHAIN), ("depth_to_space", ctypes.c_int),
                ("dtype", ctypes.c_int), ("mode", ctypes.c_int)]


class is_tokens(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("len", ctypes.c_int), ("heads", ctypes.c_int),
                ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class rotary_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("d", "rot", "axes", "layout", "scaling", "original_len")] + \
               [(f, ctypes.c_double) for f in ("base", "factor", "ramp_low", "ramp_high", "magnitude")]


class qk_norm_desc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("q", is_tokens),
                ("k", is_tokens), ("q_out", is_tokens), ("k_out", is_tokens),
                ("q_pos_batch_stride", ctypes.c_int64), ("k_pos_batch_stride", ctypes.c_int64)]


class cross_attention_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("n", "lq", "lk", "hq", "hkv", "d", "dtype")] + \
               [("scale", ctypes.c_float)] + \
               [(f, ctypes.c_int64 * 3) for f in ("q_stride", "k_stride", "v_stride", "out_stride")] + \
               [("mask_batch_stride", ctypes.c_int64)]


class is_rows(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("len", ctypes.c_int), ("batch_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64)]


class block_norm_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("dtype", "c", "norm", "post")] + \
               [("eps", ctypes.c_float), ("residual_scale", ctypes.c_float)] + \
               [(f, is_rows) for f in ("x", "y", "x_out", "out")] + \
               [(f, ctypes.c_int64) for f in ("gate_stride", "scale_stride", "shift_stride")]


class dense_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("n", "len", "in_", "features", "dtype", "activation")] + \
               [(f, ctypes.c_int64 * 2) for f in ("x_stride", "residual_stride", "out_stride")] + \
               [("w_stride", ctypes.c_int64)]


class held_states_desc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in ("n", "len", "heads", "d", "dtype")]


class held_attention_desc(ctypes.Structure):
    _fields_ = [("held", held_states_desc), ("lq", ctypes.c_int), ("hq", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3),
                ("mask_batch_stride", ctypes.c_int64)]


# (name, restype, argtypes) of every function the header declares.
_vp = ctypes.c_void_p
SIGNATURES = [
    ("conv2d_create", ctypes.c_int, [ctypes.POINTER(conv2d_desc), ctypes.POINTER(_vp)]),
    ("conv2d_forward", ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp]),
    ("conv2d_destroy", None, [_vp]),
    ("conv2d_get_plan_info", ctypes.c_int, [_vp, ctypes.POINTER(conv2d_plan_info)]),
    ("conv2d_list_variants", ctypes.c_int, [ctypes.POINTER(conv2d_desc), ctypes.POINTER(conv2d_variant),
                                            ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
    ("conv2d_create_variant", ctypes.c_int, [ctypes.POINTER(conv2d_desc), ctypes.c_int, ctypes.POINTER(_vp)]),
    ("conv2d_autotune", ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int,
                                       ctypes.POINTER(conv2d_variant), ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int)]),
    ("conv_chain_workspace_size", ctypes.c_int, [ctypes.POINTER(conv_chain_desc), ctypes.POINTER(ctypes.c_size_t)]),
    ("conv_chain_forward", ctypes.c_int, [ctypes.POINTER(conv_chain_desc), _vp, ctypes.POINTER(_vp),
                                          ctypes.POINTER(_vp), _vp, _vp, ctypes.c_size_t, _vp]),
    ("conv_chain_forward_noalloc", ctypes.c_int, [ctypes.POINTER(conv_chain_desc), _vp, ctypes.POINTER(_vp),
                                                  ctypes.POINTER(_vp), _vp, _vp]),
    ("conv_chain_kernel_name", ctypes.c_int, [ctypes.POINTER(conv_chain_desc), ctypes.c_char_p, ctypes.c_size_t]),
    ("conv_chain_groups", ctypes.c_int, [ctypes.POINTER(conv_chain_desc), ctypes.POINTER(ctypes.c_int), ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int)]),
    ("rotary_create", ctypes.c_int, [ctypes.POINTER(rotary_desc), ctypes.POINTER(_vp)]),
    ("rotary_destroy", None, [_vp]),
    ("rotary_get_frequencies", ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_double), ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_int)]),
    ("rotary_forward", ctypes.c_int, [_vp, ctypes.c_int, ctypes.POINTER(is_tokens), _vp, _vp, ctypes.c_int64,
                                      ctypes.POINTER(is_tokens), _vp, _vp]),
    ("qk_norm_rotary_forward", ctypes.c_int, [_vp, ctypes.POINTER(qk_norm_desc)] + [_vp] * 9),
    ("cross_attention_create", ctypes.c_int, [ctypes.POINTER(cross_attention_desc), ctypes.POINTER(_vp)]),
    ("cross_attention_destroy", None, [_vp]),
    ("cross_attention_workspace_size", ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    ("cross_attention_get_plan_info", ctypes.c_int, [_vp, ctypes.POINTER(conv2d_plan_info)]),
    ("cross_attention_forward", ctypes.c_int, [_vp] * 9 + [ctypes.c_size_t, _vp]),
    ("block_norm_forward", ctypes.c_int, [ctypes.POINTER(block_norm_desc)] + [_vp] * 11),
    ("dense_create", ctypes.c_int, [ctypes.POINTER(dense_desc), ctypes.POINTER(_vp)]),
    ("dense_destroy", None, [_vp]),
    ("dense_workspace_size", ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    ("dense_get_plan_info", ctypes.c_int, [_vp, ctypes.POINTER(conv2d_plan_info)]),
    ("dense_forward", ctypes.c_int, [_vp] * 7 + [ctypes.c_size_t, _vp]),
    ("held_states_size", ctypes.c_int, [ctypes.POINTER(held_states_desc), ctypes.POINTER(ctypes.c_size_t)]),
    ("held_store", ctypes.c_int, [ctypes.POINTER(held_states_desc), ctypes.POINTER(is_tokens), _vp,
                                  ctypes.POINTER(is_tokens), _vp, _vp, ctypes.c_int64, _vp, ctypes.c_int, _vp,
                                  ctypes.c_size_t, _vp]),
    ("held_load", ctypes.c_int, [ctypes.POINTER(held_states_desc), _vp, ctypes.c_size_t, ctypes.c_int,
                                 ctypes.POINTER(is_tokens), _vp, ctypes.POINTER(is_tokens), _vp, _vp]),
    ("held_attention_create", ctypes.c_int, [ctypes.POINTER(held_attention_desc), ctypes.POINTER(_vp)]),
    ("held_attention_destroy", None, [_vp]),
    ("held_attention_workspace_size", ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_size_t)]),
    ("held_attention_get_plan_info", ctypes.c_int, [_vp, ctypes.POINTER(conv2d_plan_info)]),
    ("held_attention_forward", ctypes.c_int, [_vp, _vp, _vp, ctypes.c_size_t] + [_vp] * 5 + [ctypes.c_size_t, _vp]),
    ("is_lds_tile_bytes", ctypes.c_size_t, [ctypes.c_int] * 6),
    ("is_swizzle_col", ctypes.c_int, [ctypes.c_int] * 5),
    ("is_persistent_grid", ctypes.c_int, [ctypes.c_int, ctypes.c_int]),
    ("is_status_str", ctypes.c_char_p, [ctypes.c_int]),
    ("is_last_hip_error", ctypes.c_int, []),
    ("is_version", ctypes.c_int, []),
]

_lib = None


def load():
    """Open libimgstencil.so and declare every signature; raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libimgstencil.so is not built (%s); run __graft_entry__.build() "
                               "or python image_stencil_amd/build.py" % LIB_PATH)
        # Let torch load its HIP runtime first when it is installed: the library
        # then binds to that same libamdhip64.so.7, so that device pointers and
        # streams coming from torch are valid in it. Loaded first, the library
        # would pull in the system runtime, and torch would have to share it.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        lib = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


class ImgStencilError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        lib = load()
        msg = "%s: %s (%s)" % (where, STATUS_NAMES.get(status, status), lib.is_status_str(status).decode())
        if status == IS_ERR_HIP:
            msg += ", hipError_t %d" % lib.is_last_hip_error()
        super().__init__(msg)


def check(status, where):
    if status != IS_OK:
        raise ImgStencilError(status, where)
