"""Python binding of libhashattn.so (ctypes; argument marshalling only).

Every function here has the name of the C entry point it calls and forwards
device pointers taken from torch tensors plus the current CUDA stream. No step
of the computation runs in Python or torch. Loading fails loudly when the
library has not been built: there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import struct

from ._build import LIB_PATH

HA_OK = 0
HA_ERR_INVALID_ARG = -1
HA_ERR_UNSUPPORTED = -2
HA_ERR_WORKSPACE = -3
HA_ERR_CUDA = -4
HA_ERR_DEVICE = -5
HA_ERR_TIMEOUT = -6

HA_F32 = 0
HA_BF16 = 1

HA_DEVERR_SEQLEN = 0x1
HA_DEVERR_BUDGET = 0x2
HA_DEVERR_INDEX = 0x4
HA_DEVERR_COUNT = 0x8
HA_DEVERR_TIMEOUT = 0x10
HA_DEVERR_STATE = 0x20
HA_DEVERR_PAGES = 0x40

HA_NBINS = 33
HA_NOALLOC_SCRATCH_BYTES = 16 << 20

# Entry points declared in include/hashattn.h (checked by the tests).
EXPORTED = [
    "hash_attn_workspace_size", "hash_attn_workspace_init", "hash_attn_select_capacity",
    "hash_attn_decode", "hash_attn_decode_ex", "hash_attn_decode_timed", "hash_attn_decode_host",
    "hash_attn_host_staging_size", "hash_attn_score", "hash_attn_select",
    "hash_attn_select_ex", "hash_attn_workspace_size_ex", "hash_attn_selection_plan", "hash_attn_decode_path",
    "hash_attn_gather_att", "hash_attn_gather_att_noalloc", "hash_attn_merge", "hash_attn_merge_n",
    "hash_attn_encode_queries", "hash_attn_encode_keys", "hash_attn_encode_queries_mlp",
    "hash_attn_encode_keys_mlp", "hash_attn_decode_mapped", "hash_attn_topk_exact_workspace_size",
    "hash_attn_topk_exact", "hash_attn_topk_exact_timed", "hash_attn_recall",
    "hash_attn_append", "hash_attn_packed_workspace_size", "hash_attn_prefill", "hash_attn_chunk",
    "hash_attn_plan_pages", "hash_attn_append_axes", "hash_attn_prefill_ex", "hash_attn_chunk_ex",
    "hash_attn_device_status",
    "hash_attn_status_string", "hash_attn_last_error",
]


class HASelectOpts(ctypes.Structure):
    """Mirror of ``ha_select_opts``."""

    _fields_ = [("m_per_head", ctypes.c_void_p), ("exclusive_windows", ctypes.c_int32),
                ("code_words", ctypes.c_int32), ("reserved", ctypes.c_int32 * 2)]


def select_opts(m_per_head=None, exclusive_windows=False, code_words=1) -> HASelectOpts:
    o = HASelectOpts()
    o.m_per_head = _ptr(m_per_head)
    o.exclusive_windows = 1 if exclusive_windows else 0
    o.code_words = int(code_words)
    return o


class HAMlp(ctypes.Structure):
    """Mirror of ``ha_mlp`` (the MLP signature map's weights, device pointers)."""

    _fields_ = [("W1", ctypes.c_void_p), ("b1", ctypes.c_void_p), ("W2", ctypes.c_void_p),
                ("b2", ctypes.c_void_p), ("W3", ctypes.c_void_p), ("b3", ctypes.c_void_p),
                ("hidden", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def mlp(W1, b1, W2, b2, W3, b3) -> HAMlp:
    """HAMlp over float32 device tensors W1 [h_kv, H, d], b1 [h_kv, H], W2 [h_kv, H, H],
    b2 [h_kv, H], W3 [h_kv, 32, H], b3 [h_kv, 32]. The struct holds raw pointers:
    keep the tensors alive while it is used."""
    m = HAMlp()
    m.W1, m.b1, m.W2, m.b2, m.W3, m.b3 = (_ptr(t) for t in (W1, b1, W2, b2, W3, b3))
    m.hidden = int(W1.shape[1])
    return m


class HAMap(ctypes.Structure):
    """Mirror of ``ha_map``: exactly one of W (sign projection) and mlp."""

    _fields_ = [("W", ctypes.c_void_p), ("mlp", ctypes.POINTER(HAMlp))]


def sign_map(W) -> HAMap:
    m = HAMap()
    m.W = _ptr(W)
    return m


def mlp_map(weights: HAMlp) -> HAMap:
    m = HAMap()
    m.mlp = ctypes.pointer(weights)
    return m


class HAShape(ctypes.Structure):
    """Mirror of ``ha_shape`` (all strides in elements)."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("n_cap", ctypes.c_int32),
        ("q_dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
        ("q_sb", ctypes.c_int64), ("q_sh", ctypes.c_int64),
        ("k_sb", ctypes.c_int64), ("k_sh", ctypes.c_int64), ("k_sn", ctypes.c_int64),
        ("v_sb", ctypes.c_int64), ("v_sh", ctypes.c_int64), ("v_sn", ctypes.c_int64),
        ("ks_sb", ctypes.c_int64), ("ks_sh", ctypes.c_int64),
    ]


class HATokens(ctypes.Structure):
    """Mirror of ``ha_tokens`` (packed new tokens; strides in elements)."""

    _fields_ = [
        ("n_seq", ctypes.c_int32), ("total", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("q_st", ctypes.c_int64), ("q_sh", ctypes.c_int64), ("k_st", ctypes.c_int64), ("k_sh", ctypes.c_int64),
        ("v_st", ctypes.c_int64), ("v_sh", ctypes.c_int64),
    ]


class HACache(ctypes.Structure):
    """Mirror of ``ha_cache`` (a paged KV cache; strides in elements)."""

    _fields_ = [
        ("dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("table_st", ctypes.c_int64),
        ("k_sp", ctypes.c_int64), ("k_sh", ctypes.c_int64), ("k_sn", ctypes.c_int64),
        ("v_sp", ctypes.c_int64), ("v_sh", ctypes.c_int64), ("v_sn", ctypes.c_int64),
        ("ks_sp", ctypes.c_int64), ("ks_sh", ctypes.c_int64),
    ]


class HARope(ctypes.Structure):
    """Mirror of ``ha_rope``."""

    tensor = None  # inv_freq, where it came as one (see rope)
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class HARopeAxes(ctypes.Structure):
    """Mirror of ``ha_rope_axes``."""

    tensor = None  # inv_freq, where it came as one (see rope_axes)
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("reserved", ctypes.c_int32), ("axis", ctypes.c_uint8 * 64)]


class HAScoreOpts(ctypes.Structure):
    """Mirror of ``ha_score_opts``."""

    tensors = None  # slopes, prefix and first, where any of them came as a tensor (see score_opts)
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p), ("first", ctypes.c_void_p)]


class HAPaging(ctypes.Structure):
    """Mirror of ``ha_paging``."""

    _fields_ = [("n_seq", ctypes.c_int32), ("total", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("table_st", ctypes.c_int64)]


class HashAttnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{status_string(status)} ({status}): {detail}")
        self.status = status
        self.detail = detail


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded library (raises if libhashattn.so has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libhashattn.so not built at {LIB_PATH}; run __graft_entry__.build() "
                          "or python long_context_sparse_score_gb300/_build.py")
    L = ctypes.CDLL(LIB_PATH)
    SP = ctypes.POINTER(HAShape)
    L.hash_attn_workspace_size.argtypes = [SP, _I32, _I32, _I32, ctypes.POINTER(_SZ)]
    L.hash_attn_workspace_init.argtypes = [_P, _SZ, _P]
    L.hash_attn_select_capacity.argtypes = [_I32, _I32, _I32, _I32]
    L.hash_attn_select_capacity.restype = _I32
    dec = [SP, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P]
    L.hash_attn_decode.argtypes = dec
    OP = ctypes.POINTER(HASelectOpts)
    L.hash_attn_decode_ex.argtypes = dec[:11] + [OP] + dec[11:]
    L.hash_attn_select_ex.argtypes = [SP, _P, _P, _P, _P, _I32, _I32, _I32, OP, _P, _P, _P, _SZ, _P]
    L.hash_attn_workspace_size_ex.argtypes = [SP, _I32, _I32, _I32, OP, ctypes.POINTER(_SZ)]
    L.hash_attn_decode_timed.argtypes = dec + [ctypes.POINTER(_P)]
    IP = ctypes.POINTER(_I32)
    L.hash_attn_selection_plan.argtypes = [SP, _I32, IP, IP, IP, IP]
    L.hash_attn_decode_path.argtypes = [SP, _I32, _P, OP, _I32, IP]
    L.hash_attn_host_staging_size.argtypes = [SP, ctypes.POINTER(_SZ)]
    L.hash_attn_decode_host.argtypes = [SP, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P, _SZ,
                                        _P]
    L.hash_attn_score.argtypes = [SP, _P, _P, _P, _P, _P, _P, _SZ, _P]
    L.hash_attn_select.argtypes = [SP, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P]
    L.hash_attn_gather_att.argtypes = [SP, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _SZ, _P]
    L.hash_attn_gather_att_noalloc.argtypes = [SP, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _P, _P]
    L.hash_attn_merge.argtypes = [_P, _P, _P, _P, _P, _P, _I32, _I32, _P]
    L.hash_attn_merge_n.argtypes = [_P, ctypes.c_int64, _P, ctypes.c_int64, _I32, _P, _P, _I32, _I32, _P]
    L.hash_attn_encode_queries.argtypes = [SP, _P, _P, _P, _P]
    L.hash_attn_encode_keys.argtypes = [SP, _P, _P, _P, _P, _P, _P]
    L.hash_attn_encode_queries_mlp.argtypes = [SP, _P, ctypes.POINTER(HAMlp), _P, _P]
    L.hash_attn_encode_keys_mlp.argtypes = [SP, _P, ctypes.POINTER(HAMlp), _P, _P, _P, _P]
    L.hash_attn_decode_mapped.argtypes = [SP, _P, ctypes.POINTER(HAMap), _P, _P, _P, _P, _P, _P, _P, _I32, _I32,
                                          _I32, OP, _P, _P, _P, _P, _P, _SZ, _P, _P]
    L.hash_attn_topk_exact_workspace_size.argtypes = [SP, ctypes.POINTER(_SZ)]
    L.hash_attn_topk_exact.argtypes = [SP, _P, _P, _P, _I32, _P, _I32, _P, _P, _SZ, _P]
    L.hash_attn_topk_exact_timed.argtypes = [SP, _P, _P, _P, _I32, _P, _I32, _P, _P, _SZ, _P, ctypes.POINTER(_P)]
    L.hash_attn_recall.argtypes = [_P, _P, _I32, _P, _P, _I32, _I32, _P, _P]
    TP, CP = ctypes.POINTER(HATokens), ctypes.POINTER(HACache)
    L.hash_attn_append.argtypes = [TP, CP, ctypes.POINTER(HARope)] + [_P] * 13
    L.hash_attn_append_axes.argtypes = [TP, CP, ctypes.POINTER(HARopeAxes), _P, ctypes.c_int64] + [_P] * 13
    L.hash_attn_plan_pages.argtypes = [ctypes.POINTER(HAPaging)] + [_P] * 11
    L.hash_attn_packed_workspace_size.argtypes = [TP, ctypes.POINTER(_SZ)]
    L.hash_attn_prefill.argtypes = [TP] + [_P] * 7 + [_SZ, _P]
    L.hash_attn_chunk.argtypes = [TP, CP] + [_P] * 9 + [_SZ, _P]
    XP = ctypes.POINTER(HAScoreOpts)
    L.hash_attn_prefill_ex.argtypes = [TP, XP] + [_P] * 7 + [_SZ, _P]
    L.hash_attn_chunk_ex.argtypes = [TP, CP, XP] + [_P] * 9 + [_SZ, _P]
    L.hash_attn_device_status.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint32)]
    L.hash_attn_status_string.argtypes = [_I32]
    L.hash_attn_status_string.restype = ctypes.c_char_p
    L.hash_attn_last_error.argtypes = []
    L.hash_attn_last_error.restype = ctypes.c_char_p
    for name in EXPORTED:
        if name not in ("hash_attn_select_capacity", "hash_attn_status_string", "hash_attn_last_error"):
            getattr(L, name).restype = _I32
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().hash_attn_status_string(status).decode()


def last_error() -> str:
    return lib().hash_attn_last_error().decode()


def _check(status: int) -> None:
    if status != HA_OK:
        raise HashAttnError(status, last_error())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _raw_stream(device: int) -> int:
    """The current stream of a device, without building a torch.cuda.Stream (2.8 us)."""
    global _raw_stream
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _device() -> int:
    global _device
    import torch
    device = torch.cuda.current_device()  # initialises CUDA
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return device


def _stream(stream) -> int | None:
    if stream is None:
        return _raw_stream(_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _here(device: int, *tensors) -> list:
    """Addresses of the arguments (tensors, raw addresses or None); a tensor that is not
    on the current device, whose stream the call uses, is refused."""
    return [t if t is None or t.__class__ is int else t.data_ptr() if t.get_device() == device else _elsewhere(t) for t in tensors]


def _elsewhere(t):
    raise ValueError(f"tensor on {t.device}: every argument must be on the current CUDA device")


def _types() -> tuple:
    """float32, torch's types of HA_F32 and HA_BF16, those of a 32-bit integer (kept once torch is there)."""
    global _types
    import torch
    types = (torch.float32, (torch.float32, torch.bfloat16), (torch.int32, torch.uint32))
    _types = lambda: types  # noqa: E731
    return types


# What a call reads and writes goes by its descriptors, so a tensor that is smaller, or laid out
# otherwise, than the one a descriptor was made from would be read or written past its end. The
# checks below take a tensor as the descriptor tells of it; raw addresses are the caller's word.
# A call first looks at everything in one expression (what is not a tensor ends it with an
# AttributeError), and only where that fails at one thing after the other, to say what is wrong:
# 1 us less of a call's 8 (the rest of the checks' 2 is torch's own, for shapes, strides and types).
# The same for the devices and addresses (0.6 us of 1.8).
_fields_of_tokens = struct.Struct("8i6q").unpack_from
_fields_of_cache = struct.Struct("4i9q").unpack_from
_fields_of_paging = struct.Struct("6iq").unpack_from


def _whole(*specs) -> None:
    """(tensor, elements, type, name): contiguous tensors."""
    for t, n, dtype, what in specs:
        if t is not None and t.__class__ is not int and (t.numel() != n or t.dtype is not dtype or not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous, with {n} elements of {dtype}")


def _int32s(*specs) -> None:
    """(tensor, least elements, name): contiguous 32-bit integers."""
    ints = _types()[2]
    for t, n, what in specs:
        if t is not None and t.__class__ is not int and (t.numel() < n or t.dtype not in ints or not t.is_contiguous()):
            raise ValueError(f"{what} must be contiguous int32 with at least {n} elements")


def _as_made(*specs) -> None:
    """(tensor, shape, strides, type, name): tensors of this shape, type and strides (those of
    extents over 1)."""
    for t, shape, strides, dtype, what in specs:
        if t is None or t.__class__ is int or (t.shape == shape and t.stride() == strides and t.dtype is dtype):
            continue
        if t.shape != shape or t.dtype is not dtype or (0 not in shape and any(
                n > 1 and a != b for n, a, b in zip(shape, t.stride(), strides))):
            raise ValueError(f"{what} is {tuple(t.shape)} of {t.dtype} with strides {t.stride()}: its descriptor was made "
                             f"for {shape} of {dtype} with strides {strides}")


def _table_as_made(t, n: int, pages: int, stride: int) -> None:
    if t is None or t.__class__ is int:
        return
    rows, cols = t.shape
    if rows < n:
        raise ValueError(f"page_table must have a row for each of the {n} sequences")
    a, b = t.stride()
    if cols < pages or (b != 1 and pages > 1) or (a != stride and n > 1) or t.dtype not in _types()[2]:
        raise ValueError(f"page_table must be int32 with {pages} entries a row, its rows {stride} apart")


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return HA_F32
    if t.dtype == torch.bfloat16:
        return HA_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def make_shape(q, K, V, k_sig=None, *, n_cap=None, batch=None, share_kv=None) -> HAShape:
    """ha_shape from tensors: q [B, Hq, d], K/V [Bk, Hkv, n_cap, d], k_sig [Bk, Hkv, n_cap].

    A batch extent of 1 in K/V/k_sig with B > 1 is read as one cache shared by
    every batch entry (batch stride 0).
    """
    B, Hq, d = q.shape
    Bk, Hkv, ncap, dk = K.shape
    assert dk == d and V.shape == K.shape
    s = HAShape()
    s.batch, s.h_q, s.h_kv, s.d, s.n_cap = B, Hq, Hkv, d, ncap if n_cap is None else n_cap
    s.q_dtype, s.kv_dtype = _dtype_code(q), _dtype_code(K)
    s.q_sb, s.q_sh = q.stride(0), q.stride(1)
    shared = (Bk == 1 and B > 1) if share_kv is None else share_kv
    s.k_sb = 0 if shared else K.stride(0)
    s.k_sh, s.k_sn = K.stride(1), K.stride(2)
    s.v_sb = 0 if shared else V.stride(0)
    s.v_sh, s.v_sn = V.stride(1), V.stride(2)
    if k_sig is not None:
        s.ks_sb = 0 if (k_sig.shape[0] == 1 and B > 1) else k_sig.stride(0)
        s.ks_sh = k_sig.stride(1)
    return s


def hash_attn_workspace_size(shape: HAShape, m_max: int, n_sink: int, n_local: int) -> int:
    out = _SZ(0)
    _check(lib().hash_attn_workspace_size(ctypes.byref(shape), m_max, n_sink, n_local, ctypes.byref(out)))
    return out.value


def hash_attn_workspace_init(workspace, stream=None) -> None:
    _check(lib().hash_attn_workspace_init(_ptr(workspace), workspace.nbytes,
                                          _stream(stream)))


def hash_attn_select_capacity(n_cap: int, m: int, n_sink: int, n_local: int) -> int:
    return lib().hash_attn_select_capacity(n_cap, m, n_sink, n_local)


def _ws(workspace):
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def hash_attn_decode(shape, q, q_sig, k_sig, K, V, seq_lens, m_per_seq, m, n_sink, n_local,
                     out, lse, sel_idx=None, sel_cnt=None, *, workspace, stream=None) -> None:
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_decode(ctypes.byref(shape), _ptr(q), _ptr(q_sig), _ptr(k_sig), _ptr(K),
                                  _ptr(V), _ptr(seq_lens), _ptr(m_per_seq), m, n_sink, n_local,
                                  _ptr(out), _ptr(lse), _ptr(sel_idx), _ptr(sel_cnt), ws, nb,
                                  _stream(stream)))


def hash_attn_host_staging_size(shape) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().hash_attn_host_staging_size(ctypes.byref(shape), ctypes.byref(out)))
    return out.value


def hash_attn_decode_host(shape, q_host, q_sig_host, seq_lens_host, m_per_seq_host, k_sig, K, V, m, n_sink, n_local,
                          out_host, lse_host, *, staging, workspace, stream=None) -> None:
    """hash_attn_decode with q / q_sig / seq_lens / m_per_seq and out / lse in host
    memory (pinned tensors or raw addresses), staged through the device buffer
    ``staging`` (hash_attn_host_staging_size bytes)."""
    ws, nb = _ws(workspace)
    sp, sn = _ws(staging)
    _check(lib().hash_attn_decode_host(ctypes.byref(shape), _ptr(q_host), _ptr(q_sig_host), _ptr(seq_lens_host),
                                       _ptr(m_per_seq_host), _ptr(k_sig), _ptr(K), _ptr(V), m, n_sink, n_local,
                                       _ptr(out_host), _ptr(lse_host), sp, sn, ws, nb, _stream(stream)))


def hash_attn_workspace_size_ex(shape, m_max: int, n_sink: int, n_local: int, opts) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().hash_attn_workspace_size_ex(ctypes.byref(shape), m_max, n_sink, n_local,
                                             None if opts is None else ctypes.byref(opts), ctypes.byref(out)))
    return out.value


def hash_attn_selection_plan(shape, code_words: int = 1) -> dict:
    """{"fused", "ranges", "range", "chunk"}: the selection path the library takes for a shape."""
    v = [ctypes.c_int32(0) for _ in range(4)]
    _check(lib().hash_attn_selection_plan(ctypes.byref(shape), int(code_words), *(ctypes.byref(x) for x in v)))
    return dict(zip(("fused", "ranges", "range", "chunk"), (x.value for x in v)))


# decode paths (hash_attn_decode_path)
PATHS = {1: "dense_group", 2: "dense_heads", 3: "group", 4: "fused_lists", 5: "two_kernel"}


def hash_attn_decode_path(shape, m: int, m_per_seq=None, opts=None, with_selection: bool = False) -> str:
    """The kernels a decode call with this shape, budget and options runs (a name of PATHS)."""
    out = ctypes.c_int32(0)
    _check(lib().hash_attn_decode_path(ctypes.byref(shape), int(m), _ptr(m_per_seq),
                                       None if opts is None else ctypes.byref(opts), 1 if with_selection else 0,
                                       ctypes.byref(out)))
    return PATHS[out.value]


def hash_attn_decode_ex(shape, q, q_sig, k_sig, K, V, seq_lens, m_per_seq, m, n_sink, n_local, opts,
                        out, lse, sel_idx=None, sel_cnt=None, *, workspace, stream=None) -> None:
    """``opts``: an HASelectOpts (see ``select_opts``) or None."""
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_decode_ex(ctypes.byref(shape), _ptr(q), _ptr(q_sig), _ptr(k_sig), _ptr(K), _ptr(V),
                                     _ptr(seq_lens), _ptr(m_per_seq), m, n_sink, n_local,
                                     None if opts is None else ctypes.byref(opts), _ptr(out), _ptr(lse),
                                     _ptr(sel_idx), _ptr(sel_cnt), ws, nb, _stream(stream)))


def hash_attn_decode_timed(shape, q, q_sig, k_sig, K, V, seq_lens, m_per_seq, m, n_sink, n_local,
                           out, lse, events, sel_idx=None, sel_cnt=None, *, workspace,
                           stream=None) -> None:
    """``events``: four torch.cuda.Event(enable_timing=True)."""
    ws, nb = _ws(workspace)
    arr = (_P * 4)(*[e.cuda_event for e in events])
    _check(lib().hash_attn_decode_timed(ctypes.byref(shape), _ptr(q), _ptr(q_sig), _ptr(k_sig),
                                        _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(m_per_seq), m,
                                        n_sink, n_local, _ptr(out), _ptr(lse), _ptr(sel_idx),
                                        _ptr(sel_cnt), ws, nb, _stream(stream), arr))


def hash_attn_score(shape, q_sig, k_sig, seq_lens, dist=None, hist=None, *, workspace,
                    stream=None) -> None:
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_score(ctypes.byref(shape), _ptr(q_sig), _ptr(k_sig), _ptr(seq_lens),
                                 _ptr(dist), _ptr(hist), ws, nb, _stream(stream)))


def hash_attn_select(shape, q_sig, k_sig, seq_lens, m_per_seq, m, n_sink, n_local, sel_idx, sel_cnt,
                     *, workspace, stream=None) -> None:
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_select(ctypes.byref(shape), _ptr(q_sig), _ptr(k_sig), _ptr(seq_lens),
                                  _ptr(m_per_seq), m, n_sink, n_local, _ptr(sel_idx), _ptr(sel_cnt),
                                  ws, nb, _stream(stream)))


def hash_attn_select_ex(shape, q_sig, k_sig, seq_lens, m_per_seq, m, n_sink, n_local, opts, sel_idx, sel_cnt,
                        *, workspace, stream=None) -> None:
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_select_ex(ctypes.byref(shape), _ptr(q_sig), _ptr(k_sig), _ptr(seq_lens),
                                     _ptr(m_per_seq), m, n_sink, n_local,
                                     None if opts is None else ctypes.byref(opts), _ptr(sel_idx), _ptr(sel_cnt),
                                     ws, nb, _stream(stream)))


def hash_attn_gather_att(shape, q, K, V, seq_lens, idx, idx_cap, cnt, out, lse, *, workspace,
                         stream=None) -> None:
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_gather_att(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V), _ptr(seq_lens),
                                      _ptr(idx), idx_cap, _ptr(cnt), _ptr(out), _ptr(lse), ws, nb,
                                      _stream(stream)))


def hash_attn_gather_att_noalloc(shape, q, K, V, seq_lens, idx, idx_cap, cnt, out, lse, dev_flags=None,
                                 stream=None) -> None:
    """hash_attn_gather_att without a workspace: the library's built-in scratch
    serves (for callers that may not allocate device memory)."""
    _check(lib().hash_attn_gather_att_noalloc(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(V),
                                              _ptr(seq_lens), _ptr(idx), idx_cap, _ptr(cnt), _ptr(out),
                                              _ptr(lse), _ptr(dev_flags), _stream(stream)))


def hash_attn_merge(out_a, lse_a, out_b, lse_b, out, lse, rows: int, d: int, stream=None) -> None:
    _check(lib().hash_attn_merge(_ptr(out_a), _ptr(lse_a), _ptr(out_b), _ptr(lse_b), _ptr(out),
                                 _ptr(lse), rows, d, _stream(stream)))


def hash_attn_merge_n(outs, lses, out, lse, stream=None) -> None:
    """``outs`` [nseg, rows, d] and ``lses`` [nseg, rows] float32 (rows contiguous
    within a segment; any segment stride); ``out`` [rows, d], ``lse`` [rows]."""
    nseg, rows, d = outs.shape
    if tuple(lses.shape) != (nseg, rows) or outs.stride(1) != d or outs.stride(2) != 1 or lses.stride(1) != 1:
        raise ValueError("outs must be [nseg, rows, d] with contiguous rows and lses [nseg, rows]")
    _check(lib().hash_attn_merge_n(_ptr(outs), outs.stride(0), _ptr(lses), lses.stride(0), nseg, _ptr(out),
                                   _ptr(lse), rows, d, _stream(stream)))


def hash_attn_encode_queries(shape, q, W, q_sig, stream=None) -> None:
    """q_sig[b, h] = sign-projection code of q[b, h] under W[h // G] (W float32 [h_kv, 32, d])."""
    _check(lib().hash_attn_encode_queries(ctypes.byref(shape), _ptr(q), _ptr(W), _ptr(q_sig), _stream(stream)))


def hash_attn_encode_keys(shape, K, W, pos, k_sig, dev_flags=None, stream=None) -> None:
    """k_sig[b, g, pos[b]] = code of K[b, g, pos[b]] under W[g], for pos[b] in [0, n_cap)."""
    _check(lib().hash_attn_encode_keys(ctypes.byref(shape), _ptr(K), _ptr(W), _ptr(pos), _ptr(k_sig),
                                       _ptr(dev_flags), _stream(stream)))


def hash_attn_encode_queries_mlp(shape, q, weights: HAMlp, q_sig, stream=None) -> None:
    """q_sig[b, h] = code of q[b, h] under the MLP map of KV head h / G."""
    _check(lib().hash_attn_encode_queries_mlp(ctypes.byref(shape), _ptr(q), ctypes.byref(weights), _ptr(q_sig),
                                              _stream(stream)))


def hash_attn_encode_keys_mlp(shape, K, weights: HAMlp, pos, k_sig, dev_flags=None, stream=None) -> None:
    """k_sig[b, g, pos[b]] = code of K[b, g, pos[b]] under the MLP map of KV head g."""
    _check(lib().hash_attn_encode_keys_mlp(ctypes.byref(shape), _ptr(K), ctypes.byref(weights), _ptr(pos),
                                           _ptr(k_sig), _ptr(dev_flags), _stream(stream)))


def hash_attn_decode_mapped(shape, q, map_, pos, q_sig, k_sig, K, V, seq_lens, m_per_seq, m, n_sink, n_local,
                            opts, out, lse, sel_idx=None, sel_cnt=None, *, workspace, dev_flags=None,
                            stream=None) -> None:
    """One decode step with the signature map (``sign_map`` / ``mlp_map``) ahead of SCORE."""
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_decode_mapped(ctypes.byref(shape), _ptr(q), ctypes.byref(map_), _ptr(pos), _ptr(q_sig),
                                         _ptr(k_sig), _ptr(K), _ptr(V), _ptr(seq_lens), _ptr(m_per_seq), m,
                                         n_sink, n_local, None if opts is None else ctypes.byref(opts), _ptr(out),
                                         _ptr(lse), _ptr(sel_idx), _ptr(sel_cnt), ws, nb, _ptr(dev_flags),
                                         _stream(stream)))


def hash_attn_topk_exact_workspace_size(shape) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().hash_attn_topk_exact_workspace_size(ctypes.byref(shape), ctypes.byref(out)))
    return out.value


def hash_attn_topk_exact(shape, q, K, seq_lens, m, idx, cnt, *, workspace, stream=None) -> None:
    """idx [B, Hq, cap] / cnt [B, Hq]: the min(m, n) largest <q, k_i> per head, ascending."""
    ws, nb = _ws(workspace)
    _check(lib().hash_attn_topk_exact(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(seq_lens), m, _ptr(idx),
                                      idx.shape[-1], _ptr(cnt), ws, nb, _stream(stream)))


def hash_attn_topk_exact_timed(shape, q, K, seq_lens, m, idx, cnt, events, *, workspace, stream=None) -> None:
    """hash_attn_topk_exact with ``events``: three torch.cuda.Event(enable_timing=True),
    recorded before the scores, between the scores and the top-m, and after."""
    ws, nb = _ws(workspace)
    arr = (_P * 3)(*[e.cuda_event for e in events])
    _check(lib().hash_attn_topk_exact_timed(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(seq_lens), m, _ptr(idx),
                                            idx.shape[-1], _ptr(cnt), ws, nb, _stream(stream), arr))


def hash_attn_recall(sel_idx, sel_cnt, ref_idx, ref_cnt, recall, stream=None) -> None:
    """recall[h] = |sel_h & ref_h| / |ref_h| over [heads, cap] index lists (any leading shape)."""
    heads = sel_cnt.numel()
    _check(lib().hash_attn_recall(_ptr(sel_idx), _ptr(sel_cnt), sel_idx.shape[-1], _ptr(ref_idx), _ptr(ref_cnt),
                                  ref_idx.shape[-1], heads, _ptr(recall), _stream(stream)))


def make_tokens(q, k, v, n_seq: int, *, h_kv: int | None = None, out_dtype=None) -> HATokens:
    """ha_tokens from packed tensors: q [total, Hq, d], k and v [total, Hkv, d] (None
    with ``h_kv`` where only the queries are packed). ``out_dtype``: torch.float32
    (the default) or torch.bfloat16."""
    import torch
    t = HATokens()
    t.total, t.h_q, t.d = q.shape
    t.n_seq = int(n_seq)
    t.h_kv = int(h_kv) if k is None else k.shape[1]
    t.dtype = _dtype_code(q)
    t.out_dtype = HA_BF16 if out_dtype == torch.bfloat16 else HA_F32
    if out_dtype not in (None, torch.float32, torch.bfloat16):
        raise ValueError(f"unsupported out_dtype {out_dtype}")
    t.q_st, t.q_sh = _rows(q, "q", t.dtype, (t.total, t.h_q, t.d))[:2]
    if k is not None:
        t.k_st, t.k_sh = _rows(k, "k", t.dtype, (t.total, t.h_kv, t.d))[:2]
        t.v_st, t.v_sh = _rows(v, "v", t.dtype, (t.total, t.h_kv, t.d))[:2]
    return t


def _rows(x, what, dtype, shape):
    """Strides of a tensor that must have this shape, type and contiguous rows."""
    if tuple(x.shape) != tuple(shape) or _dtype_code(x) != dtype or (x.shape[-1] > 1 and x.stride(-1) != 1):
        raise ValueError(f"{what} must be {tuple(shape)} of one dtype with contiguous rows")
    return x.stride()


def make_cache(K, V, page_table, k_sig=None) -> HACache:
    """ha_cache from pools K, V [n_pages, Hkv, page_size, d] (for [page, token, head, d]
    in memory pass ``pool.permute(0, 2, 1, 3)``), page_table int32 [n_seq, max_pages]
    and, where codes are written, k_sig [n_pages, Hkv, page_size]."""
    c = HACache()
    c.n_pages, h_kv, c.page_size, d = K.shape
    c.dtype = _dtype_code(K)
    c.k_sp, c.k_sh, c.k_sn = _rows(K, "K", c.dtype, K.shape)[:3]
    c.v_sp, c.v_sh, c.v_sn = _rows(V, "V", c.dtype, K.shape)[:3]
    if (page_table.dim() != 2 or page_table.element_size() != 4 or page_table.is_floating_point()
            or page_table.stride(1) != 1 and page_table.shape[1] > 1):
        raise ValueError("page_table must be int32 [n_seq, max_pages] with contiguous rows")
    c.max_pages, c.table_st = page_table.shape[1], page_table.stride(0)
    if k_sig is not None:
        if tuple(k_sig.shape) != tuple(K.shape[:3]) or k_sig.element_size() != 4 or k_sig.stride(2) != 1 and c.page_size > 1:
            raise ValueError("k_sig must be 32-bit [n_pages, Hkv, page_size] with contiguous rows")
        c.ks_sp, c.ks_sh = k_sig.stride(0), k_sig.stride(1)
    return c


def rope(inv_freq, interleaved: bool = False) -> HARope:
    """HARope over a contiguous float32 device tensor inv_freq [rot_dim / 2] (which it keeps)."""
    if inv_freq.dtype is not _types()[0] or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous float32")
    r = HARope()
    r.tensor = inv_freq
    r.inv_freq = _ptr(inv_freq)
    r.rot_dim = 2 * inv_freq.numel()
    r.interleaved = 1 if interleaved else 0
    return r


def _append_checked(tokens, cache, q, k, v, page_table, cu, seq_lens, q_out, K, V, W, k_sig, dev_flags) -> bool:
    f32, types, ints = _types()
    n, T, h_q, h_kv, d, dtype, _, _, q_st, q_sh, k_st, k_sh, v_st, v_sh = _fields_of_tokens(tokens)
    pool, n_pages, size, pages, table_st, K_sp, K_sh, K_sn, V_sp, V_sh, V_sn, ks_sp, ks_sh = _fields_of_cache(cache)
    dtype, pool, rows, cached = types[dtype], types[pool], (T, h_kv, d), (n_pages, h_kv, size, d)
    try:
        good = (q.shape == (T, h_q, d) and q.stride() == (q_st, q_sh, 1) and q.dtype is dtype
                and k.shape == rows and k.stride() == (k_st, k_sh, 1) and k.dtype is dtype
                and v.shape == rows and v.stride() == (v_st, v_sh, 1) and v.dtype is dtype
                and K.shape == cached and K.stride() == (K_sp, K_sh, K_sn, 1) and K.dtype is pool
                and V.shape == cached and V.stride() == (V_sp, V_sh, V_sn, 1) and V.dtype is pool
                and page_table.shape == (n, pages) and page_table.stride() == (table_st, 1) and page_table.dtype in ints
                and q_out.numel() == T * h_q * d and q_out.dtype is dtype and q_out.is_contiguous()
                and cu.numel() == n + 1 and cu.dtype in ints and cu.is_contiguous()
                and seq_lens.numel() == n and seq_lens.dtype in ints and seq_lens.is_contiguous()
                and W is None and k_sig is None and dev_flags is None)
    except AttributeError:
        good = False
    if not good:
        _whole((q_out, T * h_q * d, dtype, "q_out"), (W, h_kv * 32 * d, f32, "W"))
        _int32s((cu, n + 1, "cu"), (seq_lens, n, "seq_lens"), (dev_flags, 1, "dev_flags"))
        _as_made((q, (T, h_q, d), (q_st, q_sh, 1), dtype, "q"), (k, rows, (k_st, k_sh, 1), dtype, "k"),
                 (v, rows, (v_st, v_sh, 1), dtype, "v"), (K, cached, (K_sp, K_sh, K_sn, 1), pool, "K"),
                 (V, cached, (V_sp, V_sh, V_sn, 1), pool, "V"))
        _table_as_made(page_table, n, pages, table_st)
        if k_sig is not None and k_sig.__class__ is not int:
            _as_made((k_sig, cached[:3], (ks_sp, ks_sh, 1), k_sig.dtype if k_sig.dtype in ints else ints[0], "k_sig"))
    return good


def _append_at(good, device, q, k, v, W, page_table, cu, seq_lens, q_out, K, V, k_sig, dev_flags):
    """The addresses of an append's arguments, in the order of its C entry; ``good``: all but the optional ones are tensors."""
    if good and (device == q.get_device() == k.get_device() == v.get_device() == page_table.get_device() == cu.get_device()
                 == seq_lens.get_device() == q_out.get_device() == K.get_device() == V.get_device()):
        return (q.data_ptr(), k.data_ptr(), v.data_ptr(), None, page_table.data_ptr(), cu.data_ptr(), seq_lens.data_ptr(),
                q_out.data_ptr(), K.data_ptr(), V.data_ptr(), None, None)
    return _here(device, q, k, v, W, page_table, cu, seq_lens, q_out, K, V, k_sig, dev_flags)


def hash_attn_append(tokens, cache, q, k, v, page_table, cu, seq_lens, q_out, K, V, *, rope=None, W=None, k_sig=None,
                     dev_flags=None, stream=None) -> None:
    """Rotate the packed new tokens' q (into ``q_out``) and k by position and write k, v
    (and with ``W`` the keys' codes) into the paged cache; ``q`` and ``q_out`` may be None."""
    good = _append_checked(tokens, cache, q, k, v, page_table, cu, seq_lens, q_out, K, V, W, k_sig, dev_flags)
    device = _device()
    a = _append_at(good, device, q, k, v, W, page_table, cu, seq_lens, q_out, K, V, k_sig, dev_flags)
    if rope is not None and rope.tensor is not None and rope.tensor.get_device() != device:
        _elsewhere(rope.tensor)
    _check(lib().hash_attn_append(tokens, cache, rope, *a, _raw_stream(device) if stream is None else _stream(stream)))


def rope_axes(inv_freq, axis, interleaved: bool = False) -> HARopeAxes:
    """HARopeAxes over a contiguous float32 device tensor inv_freq [rot_dim / 2] (which it keeps);
    ``axis``: the axis of every pair (whole numbers from 0)."""
    if inv_freq.dtype is not _types()[0] or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous float32")
    axis = [int(a) for a in axis]
    if len(axis) != inv_freq.numel() or not axis or min(axis) < 0 or max(axis) > 7 or len(axis) > 64:
        raise ValueError(f"axis must give each of the {inv_freq.numel()} pairs (64 at most) one of 8 axes")
    r = HARopeAxes()
    r.tensor = inv_freq
    r.inv_freq = _ptr(inv_freq)
    r.rot_dim = 2 * len(axis)
    r.interleaved = 1 if interleaved else 0
    r.n_axes = max(axis) + 1
    r.axis[:len(axis)] = axis
    return r


def hash_attn_append_axes(tokens, cache, q, k, v, page_table, cu, seq_lens, positions, q_out, K, V, *, rope, W=None, k_sig=None,
                          dev_flags=None, stream=None) -> None:
    """hash_attn_append with rotations by several axes: ``rope`` from ``rope_axes``, ``positions``
    int32 [n_axes, total] (rows contiguous; more axes than the rope has are not read)."""
    good = _append_checked(tokens, cache, q, k, v, page_table, cu, seq_lens, q_out, K, V, W, k_sig, dev_flags)
    pos_st = T = tokens.total
    if positions.__class__ is not int:
        i32, n = _types()[2][0], rope.n_axes
        if not (positions.shape == (n, T) and positions.is_contiguous() and positions.dtype is i32):
            axes, rows = positions.shape
            pos_st = positions.stride(0)
            if (axes < n or rows != T or positions.dtype is not i32 or (positions.stride(1) != 1 and rows > 1) or (pos_st < rows and axes > 1)):
                raise ValueError(f"positions must be int32 [{n}, {T}] with contiguous rows")
    device = _device()
    at, = _here(device, positions)
    a = _append_at(good, device, q, k, v, W, page_table, cu, seq_lens, q_out, K, V, k_sig, dev_flags)
    if rope.tensor is not None and rope.tensor.get_device() != device:
        _elsewhere(rope.tensor)
    _check(lib().hash_attn_append_axes(tokens, cache, rope, at, pos_st, *a, _raw_stream(device) if stream is None else _stream(stream)))


def _int32(x, what) -> int:
    """A structure's field would keep the low 32 bits of anything else, without a word."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{what} must be a 32-bit number (got {x})")
    return x


def make_paging(page_table, n_pages: int, page_size: int, total: int) -> HAPaging:
    """ha_paging of sequences whose pages are in ``page_table`` int32 [n_seq, max_pages], out of a pool
    of ``n_pages``; ``total``: rows that the packed buffers have room for."""
    if page_table.dim() != 2 or page_table.dtype not in _types()[2] or page_table.stride(1) != 1 and page_table.shape[1] > 1:
        raise ValueError("page_table must be int32 [n_seq, max_pages] with contiguous rows")
    p = HAPaging()
    p.n_seq, p.max_pages = page_table.shape
    p.total, p.n_pages, p.page_size = _int32(total, "total"), _int32(n_pages, "n_pages"), _int32(page_size, "page_size")
    p.table_st = page_table.stride(0)
    return p


def hash_attn_plan_pages(paging, new_lens, seq_lens, seq_lens_out, cu, page_table, free_pages, n_free, n_free_out, *, slots=None,
                         dev_flags=None, stream=None) -> None:
    """Plan a step's pages: ``seq_lens_out`` and ``n_free_out`` may be ``seq_lens`` and ``n_free``; the table
    and the stack of free pages are updated in place (a plan changes neither if run again)."""
    ints = _types()[2]
    n, total, n_pages, _, pages, _, table_st = _fields_of_paging(paging)
    try:
        good = (new_lens.numel() == n and new_lens.dtype in ints and new_lens.is_contiguous()
                and seq_lens.numel() == n and seq_lens.dtype in ints and seq_lens.is_contiguous()
                and seq_lens_out.numel() == n and seq_lens_out.dtype in ints and seq_lens_out.is_contiguous()
                and cu.numel() == n + 1 and cu.dtype in ints and cu.is_contiguous()
                and page_table.shape == (n, pages) and page_table.stride() == (table_st, 1) and page_table.dtype in ints
                and free_pages.numel() == n_pages and free_pages.dtype in ints and free_pages.is_contiguous()
                and n_free.numel() == 1 and n_free.dtype in ints and n_free_out.numel() == 1 and n_free_out.dtype in ints
                and slots.numel() == total and slots.dtype in ints and slots.is_contiguous() and dev_flags is None)
    except AttributeError:
        good = False
    if not good:
        _int32s((new_lens, n, "new_lens"), (seq_lens, n, "seq_lens"), (seq_lens_out, n, "seq_lens_out"), (cu, n + 1, "cu"),
                (free_pages, n_pages, "free_pages"), (n_free, 1, "n_free"), (n_free_out, 1, "n_free_out"),
                (slots, total, "slots"), (dev_flags, 1, "dev_flags"))
        _table_as_made(page_table, n, pages, table_st)
    device = _device()
    if good and (device == new_lens.get_device() == seq_lens.get_device() == seq_lens_out.get_device() == cu.get_device()
                 == page_table.get_device() == slots.get_device() == free_pages.get_device() == n_free.get_device()
                 == n_free_out.get_device()):
        a = (new_lens.data_ptr(), seq_lens.data_ptr(), seq_lens_out.data_ptr(), cu.data_ptr(), page_table.data_ptr(),
             slots.data_ptr(), free_pages.data_ptr(), n_free.data_ptr(), n_free_out.data_ptr(), None)
    else:
        a = _here(device, new_lens, seq_lens, seq_lens_out, cu, page_table, slots, free_pages, n_free, n_free_out, dev_flags)
    _check(lib().hash_attn_plan_pages(paging, *a, _raw_stream(device) if stream is None else _stream(stream)))


def hash_attn_packed_workspace_size(tokens) -> int:
    out = _SZ(0)
    _check(lib().hash_attn_packed_workspace_size(ctypes.byref(tokens), ctypes.byref(out)))
    return out.value


def hash_attn_prefill(tokens, q, K, V, cu, out, lse, *, workspace, stream=None, _opts=None) -> None:
    """Causal attention over packed prompts; out [total, Hq, d], lse [total, Hq] contiguous."""
    f32, types, ints = _types()
    n, T, h_q, h_kv, d, dtype, out_dtype, _, q_st, q_sh, k_st, k_sh, v_st, v_sh = _fields_of_tokens(tokens)
    dtype, out_dtype, rows = types[dtype], types[out_dtype], (T, h_kv, d)
    try:
        good = (q.shape == (T, h_q, d) and q.stride() == (q_st, q_sh, 1) and q.dtype is dtype
                and K.shape == rows and K.stride() == (k_st, k_sh, 1) and K.dtype is dtype
                and V.shape == rows and V.stride() == (v_st, v_sh, 1) and V.dtype is dtype
                and out.numel() == T * h_q * d and out.dtype is out_dtype and out.is_contiguous()
                and lse.numel() == T * h_q and lse.dtype is f32 and lse.is_contiguous()
                and cu.numel() == n + 1 and cu.dtype in ints and cu.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        _whole((out, T * h_q * d, out_dtype, "out"), (lse, T * h_q, f32, "lse"))
        _int32s((cu, n + 1, "cu"))
        _as_made((q, (T, h_q, d), (q_st, q_sh, 1), dtype, "q"), (K, rows, (k_st, k_sh, 1), dtype, "K"),
                 (V, rows, (v_st, v_sh, 1), dtype, "V"))
    device = _device()
    if _opts is not None:
        _opts_checked(_opts, tokens, device)
    if good and (device == q.get_device() == K.get_device() == V.get_device() == cu.get_device() == out.get_device()
                 == lse.get_device() == workspace.get_device()):
        a = (q.data_ptr(), K.data_ptr(), V.data_ptr(), cu.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr())
    else:
        a = _here(device, q, K, V, cu, out, lse, workspace)
    if _opts is not None:
        _check(lib().hash_attn_prefill_ex(tokens, _opts, *a, workspace.nbytes,
                                          _raw_stream(device) if stream is None else _stream(stream)))
        return
    _check(lib().hash_attn_prefill(tokens, *a, workspace.nbytes,
                                   _raw_stream(device) if stream is None else _stream(stream)))


def hash_attn_chunk(tokens, cache, q, K, V, page_table, cu, seq_lens, out, lse, *, workspace, stream=None, _opts=None) -> None:
    """Attention of the packed new tokens over the paged cache (their keys are in it already)."""
    f32, types, ints = _types()
    n, T, h_q, h_kv, d, dtype, out_dtype, _, q_st, q_sh, _, _, _, _ = _fields_of_tokens(tokens)
    pool, n_pages, size, pages, table_st, K_sp, K_sh, K_sn, V_sp, V_sh, V_sn, _, _ = _fields_of_cache(cache)
    dtype, out_dtype, pool, cached = types[dtype], types[out_dtype], types[pool], (n_pages, h_kv, size, d)
    try:
        good = (q.shape == (T, h_q, d) and q.stride() == (q_st, q_sh, 1) and q.dtype is dtype
                and K.shape == cached and K.stride() == (K_sp, K_sh, K_sn, 1) and K.dtype is pool
                and V.shape == cached and V.stride() == (V_sp, V_sh, V_sn, 1) and V.dtype is pool
                and page_table.shape == (n, pages) and page_table.stride() == (table_st, 1) and page_table.dtype in ints
                and out.numel() == T * h_q * d and out.dtype is out_dtype and out.is_contiguous()
                and lse.numel() == T * h_q and lse.dtype is f32 and lse.is_contiguous()
                and cu.numel() == n + 1 and cu.dtype in ints and cu.is_contiguous()
                and seq_lens.numel() == n and seq_lens.dtype in ints and seq_lens.is_contiguous())
    except AttributeError:
        good = False
    if not good:
        _whole((out, T * h_q * d, out_dtype, "out"), (lse, T * h_q, f32, "lse"))
        _int32s((cu, n + 1, "cu"), (seq_lens, n, "seq_lens"))
        _as_made((q, (T, h_q, d), (q_st, q_sh, 1), dtype, "q"), (K, cached, (K_sp, K_sh, K_sn, 1), pool, "K"),
                 (V, cached, (V_sp, V_sh, V_sn, 1), pool, "V"))
        _table_as_made(page_table, n, pages, table_st)
    device = _device()
    if _opts is not None:
        _opts_checked(_opts, tokens, device)
    if good and (device == q.get_device() == K.get_device() == V.get_device() == page_table.get_device() == cu.get_device()
                 == seq_lens.get_device() == out.get_device() == lse.get_device() == workspace.get_device()):
        a = (q.data_ptr(), K.data_ptr(), V.data_ptr(), page_table.data_ptr(), cu.data_ptr(), seq_lens.data_ptr(),
             out.data_ptr(), lse.data_ptr(), workspace.data_ptr())
    else:
        a = _here(device, q, K, V, page_table, cu, seq_lens, out, lse, workspace)
    if _opts is not None:
        _check(lib().hash_attn_chunk_ex(tokens, cache, _opts, *a, workspace.nbytes,
                                        _raw_stream(device) if stream is None else _stream(stream)))
        return
    _check(lib().hash_attn_chunk(tokens, cache, *a, workspace.nbytes,
                                 _raw_stream(device) if stream is None else _stream(stream)))


def score_opts(*, scale: float = 0.0, softcap: float = 0.0, window: int = 0, slopes=None, prefix=None, first=None) -> HAScoreOpts:
    """HAScoreOpts: scores scale z (0: 1 / sqrt(d)), capped to softcap tanh(z / softcap), less
    slopes[h] times the distance; a sliding ``window``; keys below prefix[s] seen by every token of sequence s,
    keys before first[s] by none. ``slopes`` float32 [h_q], ``prefix`` and ``first`` int32 [n_seq], contiguous device
    tensors (which it keeps), raw addresses or None."""
    o = HAScoreOpts()
    o.scale, o.softcap, o.window = scale, softcap, _int32(window, "window")
    if (scale and not o.scale) or (softcap and not o.softcap):  # 0 would say: the default
        raise ValueError(f"scale and softcap must be 0 or float32 numbers (got {scale}, {softcap})")
    o.slopes, o.prefix, o.first = (_ptr(t) for t in (slopes, prefix, first))
    tensors = tuple(None if t.__class__ is int else t for t in (slopes, prefix, first))
    o.tensors = tensors if any(t is not None for t in tensors) else None
    return o


def _opts_checked(opts, tokens, device) -> None:
    if opts.tensors is None:
        return
    slopes, prefix, first = opts.tensors
    _whole((slopes, tokens.h_q, _types()[0], "slopes"))
    _int32s((prefix, tokens.n_seq, "prefix"), (first, tokens.n_seq, "first"))
    _here(device, slopes, prefix, first)


def hash_attn_prefill_ex(tokens, opts, q, K, V, cu, out, lse, *, workspace, stream=None) -> None:
    """hash_attn_prefill with score options (``score_opts``; None: without)."""
    hash_attn_prefill(tokens, q, K, V, cu, out, lse, workspace=workspace, stream=stream, _opts=opts)


def hash_attn_chunk_ex(tokens, cache, opts, q, K, V, page_table, cu, seq_lens, out, lse, *, workspace, stream=None) -> None:
    """hash_attn_chunk with score options (``score_opts``; None: without)."""
    hash_attn_chunk(tokens, cache, q, K, V, page_table, cu, seq_lens, out, lse, workspace=workspace, stream=stream, _opts=opts)


def hash_attn_device_status(workspace, stream=None) -> tuple[int, int]:
    """(status, raw flags); synchronises the stream and clears the error word."""
    flags = ctypes.c_uint32(0)
    st = lib().hash_attn_device_status(_ptr(workspace), _stream(stream), ctypes.byref(flags))
    return st, flags.value
