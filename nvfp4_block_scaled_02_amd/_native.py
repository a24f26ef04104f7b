"""ctypes loader for libnvfp4.so (the C ABI of include/nvfp4.h).

The library is built in-tree by ``nvfp4_block_scaled_02_amd.build`` (or
``__graft_entry__.build()``).  There is no fallback: if the library is
missing or cannot be loaded, every call raises.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")
ABI_VERSION = 9  # NVFP4_ABI_VERSION of include/nvfp4.h that these signatures follow

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_HIP = 0, 1, 2, 3
SCALE_E4M3, SCALE_UE5M3 = 0, 1
SELECT_6, SELECT_4OVER6 = 0, 1
SELECT_4OVER6_MAE, SELECT_4OVER6_MAXERR, SELECT_SWEEP = 2, 3, 4
ROUND_RNE, ROUND_SR = 0, 1
AXIS_ROW, AXIS_COL = 1, 2
TARGET_NVFP4, TARGET_MXFP8 = 0, 1

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32
_f32 = ctypes.c_float


class QuantArgs(ctypes.Structure):
    """nvfp4_quant_args of include/nvfp4.h (same field order, so the same
    C layout)."""
    _fields_ = [("x", _vp), ("rows", _i64), ("cols", _i64), ("amax", _vp),
                ("global_fp8_max", _f32), ("scale_fmt", _int), ("select", _int),
                ("rounding", _int), ("axes", _int), ("seed", _u64), ("codes", _vp),
                ("scales", _vp), ("codes_t", _vp), ("scales_t", _vp), ("count4", _vp),
                ("workspace", _vp)]


PAIRS_HALVES, PAIRS_NEIGHBOURS = 0, 1
KV_COUNTER_BYTES = 131072


class KVCacheArgs(ctypes.Structure):
    """nvfp4_kv_cache."""
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp),
                ("k_amax", _vp), ("v_amax", _vp), ("num_pages", _i64), ("kv_heads", _int),
                ("page_size", _int), ("head_dim", _int), ("global_fp8_max", _f32)]


class KVPlanArgs(ctypes.Structure):
    """nvfp4_kv_plan_args."""
    _fields_ = [("ctx_lens", _vp), ("new_lens", _vp), ("batch", _i64), ("block_table", _vp),
                ("table_width", _i64), ("free_pages", _vp), ("free_count", _vp),
                ("num_pages", _i64), ("page_size", _int), ("tokens", _i64), ("cu_new", _vp),
                ("seq_lens", _vp), ("positions", _vp), ("slots", _vp), ("free_count_out", _vp),
                ("refused", _vp)]


class QKArgs(ctypes.Structure):
    """nvfp4_qk_args."""
    _fields_ = [("q", _vp), ("k", _vp), ("tokens", _i64), ("q_heads", _int), ("k_heads", _int),
                ("head_dim", _int), ("q_stride", _i64), ("k_stride", _i64), ("positions", _vp),
                ("cos", _vp), ("sin", _vp), ("max_pos", _i64), ("rot_dim", _int), ("pairs", _int),
                ("q_weight", _vp), ("k_weight", _vp), ("eps", _f32), ("q_out", _vp),
                ("k_out", _vp), ("q_out_stride", _i64), ("k_out_stride", _i64)]


class KVAppendArgs(ctypes.Structure):
    """nvfp4_kv_append_args."""
    _fields_ = [("qk", QKArgs), ("v", _vp), ("v_stride", _i64), ("slots", _vp),
                ("cache", KVCacheArgs), ("select", _int)]


class KVAttentionArgs(ctypes.Structure):
    """nvfp4_kv_attention_args."""
    _fields_ = [("q", _vp), ("tokens", _i64), ("q_stride", _i64), ("q_heads", _int),
                ("cache", KVCacheArgs), ("block_table", _vp), ("batch", _i64),
                ("table_width", _i64), ("seq_lens", _vp), ("cu_q", _vp), ("max_seq_len", _i64),
                ("scale", _f32), ("causal", _int), ("window", _i64), ("out", _vp), ("lse", _vp),
                ("workspace", _vp), ("counters", _vp)]


_qa = ctypes.POINTER(QuantArgs)
_pa, _ka = ctypes.POINTER(KVPlanArgs), ctypes.POINTER(QKArgs)
_aa, _ta, _ca = (ctypes.POINTER(KVAppendArgs), ctypes.POINTER(KVAttentionArgs),
                 ctypes.POINTER(KVCacheArgs))
# name -> (restype, argtypes); the exported surface of include/nvfp4.h and
# include/nvfp4_testing.h (hipStream_t travels as a pointer)
SIGNATURES = {
    "nvfp4_abi_version": (_int, []),
    "nvfp4_status_string": (ctypes.c_char_p, [_int]),
    "nvfp4_workspace_bytes": (ctypes.c_size_t, []),
    "nvfp4_tensor_amax": (_int, [_vp, _i64, _vp, _vp, _vp]),
    "nvfp4_tensor_amax_noalloc": (_int, [_vp, _i64, _vp, _vp]),
    "nvfp4_quantize": (_int, [_qa, _vp]),
    "nvfp4_dequantize": (_int, [_vp, _vp, _i64, _i64, _vp, _f32, _int, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp]),
    "nvfp4_row_amax": (_int, [_vp, _i64, _i64, _vp, _vp]),
    "nvfp4_quantize_rowscaled": (_int, [_qa, _vp]),
    "nvfp4_quantize_pertoken": (_int, [_qa, _vp, _vp]),
    "nvfp4_dequantize_rowscaled": (_int, [_vp, _vp, _i64, _i64, _vp, _f32, _int, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _vp]),
    "nvfp4_quantize_2d": (_int, [_qa, _vp]),
    "nvfp4_fakequant_fwd": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "nvfp4_fakequant_bwd": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_fakequant_fwd_amax": (_int, [_vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "nvfp4_fakequant_bwd_amax": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_dequantized_amax": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _f32, _int, _vp, _vp, _vp]),
    "nvfp4_requantize_t": (_int, [_vp, _vp, _i64, _i64, _vp, _vp, _f32, _int, _int, _vp, _f32,
                                  _int, _u64, _vp, _vp, _vp]),
    "nvfp4_rht_amax": (_int, [_vp, _i64, _i64, _int, _u64, _vp, _vp, _vp]),
    "nvfp4_quantize_rht": (_int, [_qa, _u64, _vp]),
    "nvfp4_dequantize_rht": (_int, [_vp, _vp, _i64, _i64, _vp, _f32, _int, _u64, _vp, _vp]),
    "nvfp4_kv_plan": (_int, [_pa, _vp]),
    "nvfp4_qk_norm_rope": (_int, [_ka, _vp]),
    "nvfp4_qk_norm_rope_bwd_workspace_bytes": (ctypes.c_size_t, [_int]),
    "nvfp4_qk_norm_rope_bwd": (_int, [_ka, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp]),
    "nvfp4_kv_append": (_int, [_aa, _vp]),
    "nvfp4_kv_read": (_int, [_ca, _vp, _i64, _vp, _vp, _vp]),
    "nvfp4_kv_attention_workspace_bytes": (ctypes.c_size_t, [_ta]),
    "nvfp4_kv_attention": (_int, [_ta, _vp]),
    "nvfp4_test_e2m1_rne_range": (_int, [_u32, _i64, _vp, _vp]),
    "nvfp4_test_e2m1_sr": (_int, [_vp, _vp, _i64, _vp, _vp]),
    "nvfp4_test_scale_encode_range": (_int, [_int, _u32, _i64, _vp, _vp]),
    "nvfp4_test_sr_hash": (_int, [_u64, _u64, _i64, _vp, _vp]),
    "nvfp4_test_e4m3_sr": (_int, [_vp, _vp, _i64, _vp, _vp]),
}

WORKSPACE_BYTES = 66688  # NVFP4_WORKSPACE_BYTES of include/nvfp4.h

_lib = None


class NativeError(RuntimeError):
    pass


def lib():
    """The loaded library (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise NativeError(
            f"{LIB_PATH} is not built; run `python -m nvfp4_block_scaled_02_amd.build` "
            "(hipcc, gfx950) first. There is no non-native fallback.")
    l = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(l, name)
        f.restype = res
        f.argtypes = args
    if l.nvfp4_abi_version() != ABI_VERSION or l.nvfp4_workspace_bytes() != WORKSPACE_BYTES:
        raise NativeError(
            f"{LIB_PATH} has ABI version {l.nvfp4_abi_version()}, the binding expects "
            f"{ABI_VERSION}; rebuild with `python -m nvfp4_block_scaled_02_amd.build`.")
    _lib = l
    return l


def check(status, what):
    if status != OK:
        msg = lib().nvfp4_status_string(status).decode()
        raise NativeError(f"{what} failed with status {status} ({msg})")
