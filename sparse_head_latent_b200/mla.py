"""Python binding of the C ABI in include/mla.h (argument marshalling only).

Every function here forwards device pointers, sizes and the current CUDA
stream of torch to ``libmla_b200.so``; all arithmetic happens in the CUDA
kernels. There is no fallback: if the library or a CUDA device is missing,
the first call raises.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmla_b200.so")
_lock = threading.Lock()
_lib = None

MLA_ENTRY_KV_UPPROJECT, MLA_ENTRY_ATTEND, MLA_ENTRY_OUT_PROJECT, MLA_ENTRY_PREFILL, MLA_ENTRY_DECODE = 0, 1, 2, 3, 4
MLA_ENTRY_TREE_DECODE = 5
MLA_W_BF16, MLA_W_E4M3_BLOCK128 = 0, 1
MLA_PROFILE_CLASSES = 10
MLA_PATH_AUTO, MLA_PATH_BLOCK_DENSE, MLA_PATH_ABSORBED = 0, 1, 2
MLA_ACT_BF16, MLA_ACT_E4M3_DYNAMIC = 0, 1
PROFILE_CLASS_NAMES = ("topk_prepass", "weight_dequant", "gemm_kvb", "attention", "gemm_wo", "row_lists",
                       "gemm_absorb", "attention_absorbed", "act_quant", "gemm_wo_split_sum")
D_NOPE, D_ROPE, D_V, D_LATENT, D_MODEL = 128, 64, 128, 512, 7168
MLA_ROPE_INTERLEAVED, MLA_ROPE_HALF = 0, 1
MLA_ROPE_UNSCALED, MLA_ROPE_LINEAR, MLA_ROPE_YARN = 0, 1, 2
MLA_MAX_TREE = 64


class MlaDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("d_nope", ctypes.c_int), ("d_rope", ctypes.c_int), ("d_v", ctypes.c_int),
                ("d_latent", ctypes.c_int), ("d_model", ctypes.c_int),
                ("topk", ctypes.c_int), ("wdtype", ctypes.c_int), ("path", ctypes.c_int), ("act", ctypes.c_int)]


class MlaRopeTable(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_uint64 * (D_ROPE // 2)), ("magnitude", ctypes.c_float), ("layout", ctypes.c_int)]


class MlaPages(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("table_width", ctypes.c_int),
                ("layers", ctypes.c_int)]


class MlaError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: status {status} ({mla_status_str(status)})")
        self.status = status


# Exported symbols with their C signatures (checked by the tests).
_VP, _SZ = ctypes.c_void_p, ctypes.c_size_t
SIGNATURES = {
    "mla_workspace_bytes": (_SZ, [ctypes.POINTER(MlaDims), ctypes.c_int, ctypes.c_int]),
    "mla_kv_upproject": (ctypes.c_int, [ctypes.POINTER(MlaDims), _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "mla_attend": (ctypes.c_int, [ctypes.POINTER(MlaDims), _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_float,
                                  _VP, _VP, _SZ, _VP]),
    "mla_out_project": (ctypes.c_int, [ctypes.POINTER(MlaDims), _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "mla_prefill": (ctypes.c_int, [ctypes.POINTER(MlaDims), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                   ctypes.c_float, _VP, _VP, _SZ, _VP]),
    "mla_decode": (ctypes.c_int, [ctypes.POINTER(MlaDims), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                  ctypes.c_float, _VP, _VP, _SZ, _VP]),
    "mla_attend_static": (ctypes.c_int, [ctypes.POINTER(MlaDims), _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_float,
                                         _VP, _VP]),
    "mla_quantize_act": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.c_int, _VP, _VP, _VP]),
    "mla_rope_init": (ctypes.c_int, [ctypes.POINTER(MlaRopeTable), ctypes.c_int, ctypes.c_double, ctypes.c_int,
                                     ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                     ctypes.c_float]),
    "mla_rope": (ctypes.c_int, [ctypes.POINTER(MlaRopeTable), _VP, ctypes.c_longlong, ctypes.c_longlong, _VP,
                                ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                ctypes.c_int, _VP, ctypes.c_int, _VP]),
    "mla_cache_append": (ctypes.c_int, [ctypes.POINTER(MlaRopeTable), _VP, ctypes.c_longlong, _VP, ctypes.c_int,
                                        ctypes.c_float, _VP, _VP, ctypes.c_int, _VP, _VP, ctypes.c_longlong, _VP]),
    "mla_tree_decode": (ctypes.c_int, [ctypes.POINTER(MlaDims), ctypes.POINTER(MlaPages), _VP, _VP, _VP, _VP, _VP,
                                       _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _SZ, _VP]),
    "mla_cache_compact": (ctypes.c_int, [ctypes.POINTER(MlaPages), _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int,
                                         ctypes.c_int, _VP]),
    "mla_cache_copy_pages": (ctypes.c_int, [ctypes.POINTER(MlaPages), _VP, _VP, _VP, _VP, ctypes.c_int, _VP]),
    "mla_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "mla_device_status": (ctypes.c_int, [_VP, ctypes.POINTER(ctypes.c_int)]),
    "mla_set_e4m3_weight_conversion": (ctypes.c_int, [ctypes.c_int]),
    "mla_set_wait_timeout_ns": (ctypes.c_int, [ctypes.c_ulonglong]),
    "mla_test_withhold_attention_loads": (ctypes.c_int, [ctypes.c_int]),
    "mla_test_wo_split_plan": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "mla_profile_begin": (ctypes.c_int, []),
    "mla_profile_end": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int)]),
}


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Loads libmla_b200.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(f"CUDA library not built: {_LIB_PATH} is missing "
                                   "(run python -m sparse_head_latent_b200.build)")
            lib = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(lib, name)
                f.restype, f.argtypes = res, args
            _lib = lib
    return _lib


def mla_status_str(status: int) -> str:
    return load_library().mla_status_str(int(status)).decode()


def _check(fn, rc):
    if rc != 0:
        raise MlaError(fn, rc)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_dims(B, T, H, topk=0, fp8=False, path=MLA_PATH_AUTO, act=MLA_ACT_BF16) -> MlaDims:
    return MlaDims(int(B), int(T), int(H), D_NOPE, D_ROPE, D_V, D_LATENT, D_MODEL, int(topk),
                   MLA_W_E4M3_BLOCK128 if fp8 else MLA_W_BF16, int(path), int(act))


def _wtype(w: torch.Tensor) -> bool:
    if w.dtype == torch.uint8:
        return True
    if w.dtype == torch.bfloat16:
        return False
    raise ValueError("weights must be bf16 or uint8 (e4m3 codes)")


def mla_workspace_bytes(dims: MlaDims, entry: int, has_topk: bool) -> int:
    return int(load_library().mla_workspace_bytes(ctypes.byref(dims), int(entry), 1 if has_topk else 0))


def _new(shape, dtype, device, stream, returned=True):
    """An uninitialised tensor for a call on `stream` (None: the current one). The caching allocator hands out a block
    again as soon as it is freed, ordered with the block's own stream only, so the tensor comes from the pool of the
    stream that writes it: from the current stream's, it could still be in use there. `returned`: the caller gets it,
    on the current stream, whose work must then be done before the block is handed out again."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _workspace(dims, entry, has_topk, workspace, device, stream):
    need = mla_workspace_bytes(dims, entry, has_topk)
    if workspace is None:
        workspace = _new(max(need, 1), torch.uint8, device, stream, returned=False)
    return workspace, workspace.numel() * workspace.element_size()


def mla_kv_upproject(kv_latent, W_kvb, W_kvb_scale=None, kvh_out=None, workspace=None, stream=None,
                     act=MLA_ACT_BF16):
    """kv_latent bf16 [..., 512] -> kvh bf16 [rows, H*256]."""
    rows = kv_latent.numel() // D_LATENT
    H = W_kvb.shape[0] // (D_NOPE + D_V)
    dims = make_dims(1, rows, H, 0, _wtype(W_kvb), act=act)
    if kvh_out is None:
        kvh_out = _new((rows, H * (D_NOPE + D_V)), torch.bfloat16, kv_latent.device, stream)
    ws, nbytes = _workspace(dims, MLA_ENTRY_KV_UPPROJECT, False, workspace, kv_latent.device, stream)
    lib = load_library()
    _check("mla_kv_upproject", lib.mla_kv_upproject(ctypes.byref(dims), _ptr(kv_latent), _ptr(W_kvb),
                                                    _ptr(W_kvb_scale), _ptr(kvh_out), _ptr(ws), nbytes,
                                                    _stream(stream)))
    return kvh_out


def mla_attend(q, kv_latent, k_pe, W_kvb, W_kvb_scale=None, topk_idx=None, scale=192 ** -0.5,
               attn_out=None, workspace=None, stream=None, path=MLA_PATH_AUTO, act=MLA_ACT_BF16):
    """q [B,T,H,192], kv_latent [B,T,512], k_pe [B,T,64] (bf16) -> attn bf16 [B,T,H,128]."""
    B, T, H, _ = q.shape
    topk = 0 if topk_idx is None else topk_idx.shape[-1]
    dims = make_dims(B, T, H, topk, _wtype(W_kvb), path, act)
    if topk_idx is not None and topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32")
    if attn_out is None:
        attn_out = _new((B, T, H, D_V), torch.bfloat16, q.device, stream)
    ws, nbytes = _workspace(dims, MLA_ENTRY_ATTEND, topk_idx is not None, workspace, q.device, stream)
    lib = load_library()
    _check("mla_attend", lib.mla_attend(ctypes.byref(dims), _ptr(q), _ptr(kv_latent), _ptr(k_pe), _ptr(W_kvb),
                                        _ptr(W_kvb_scale), _ptr(topk_idx), float(scale), _ptr(attn_out),
                                        _ptr(ws), nbytes, _stream(stream)))
    return attn_out


MLA_STATIC_SCRATCH_BYTES = 32 << 20


def mla_attend_static(q, kv_latent, k_pe, W_kvb, W_kvb_scale=None, topk_idx=None, scale=192 ** -0.5,
                      attn_out=None, stream=None, path=MLA_PATH_AUTO, act=MLA_ACT_BF16):
    """mla_attend with the library's built-in scratch instead of a workspace,
    for callers that cannot allocate device memory; problems whose scratch
    exceeds MLA_STATIC_SCRATCH_BYTES are rejected (MlaError, status 8)."""
    B, T, H, _ = q.shape
    topk = 0 if topk_idx is None else topk_idx.shape[-1]
    dims = make_dims(B, T, H, topk, _wtype(W_kvb), path, act)
    if topk_idx is not None and topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32")
    if attn_out is None:
        attn_out = _new((B, T, H, D_V), torch.bfloat16, q.device, stream)
    _check("mla_attend_static", load_library().mla_attend_static(
        ctypes.byref(dims), _ptr(q), _ptr(kv_latent), _ptr(k_pe), _ptr(W_kvb), _ptr(W_kvb_scale), _ptr(topk_idx),
        float(scale), _ptr(attn_out), _stream(stream)))
    return attn_out


def mla_out_project(attn, W_o, W_o_scale=None, out=None, workspace=None, stream=None, act=MLA_ACT_BF16):
    """attn bf16 [rows, H*128] (or [B,T,H,128]) -> out bf16 [rows, 7168]."""
    H = W_o.shape[0] // D_V
    rows = attn.numel() // (H * D_V)
    dims = make_dims(1, rows, H, 0, _wtype(W_o), act=act)
    if out is None:
        out = _new((rows, D_MODEL), torch.bfloat16, attn.device, stream)
    ws, nbytes = _workspace(dims, MLA_ENTRY_OUT_PROJECT, False, workspace, attn.device, stream)
    lib = load_library()
    _check("mla_out_project", lib.mla_out_project(ctypes.byref(dims), _ptr(attn), _ptr(W_o), _ptr(W_o_scale),
                                                  _ptr(out), _ptr(ws), nbytes, _stream(stream)))
    return out


def mla_prefill(q, kv_latent, k_pe, W_kvb, W_o, W_kvb_scale=None, W_o_scale=None, topk_idx=None,
                scale=192 ** -0.5, out=None, workspace=None, stream=None, path=MLA_PATH_AUTO, act=MLA_ACT_BF16):
    """The whole attend block: -> out bf16 [B, T, 7168]."""
    B, T, H, _ = q.shape
    topk = 0 if topk_idx is None else topk_idx.shape[-1]
    fp8 = _wtype(W_kvb)
    if _wtype(W_o) != fp8:
        raise ValueError("W_kvb and W_o must use the same storage type")
    if topk_idx is not None and topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32")
    dims = make_dims(B, T, H, topk, fp8, path, act)
    if out is None:
        out = _new((B, T, D_MODEL), torch.bfloat16, q.device, stream)
    ws, nbytes = _workspace(dims, MLA_ENTRY_PREFILL, topk_idx is not None, workspace, q.device, stream)
    lib = load_library()
    _check("mla_prefill", lib.mla_prefill(ctypes.byref(dims), _ptr(q), _ptr(kv_latent), _ptr(k_pe), _ptr(W_kvb),
                                          _ptr(W_kvb_scale), _ptr(W_o), _ptr(W_o_scale), _ptr(topk_idx),
                                          float(scale), _ptr(out), _ptr(ws), nbytes, _stream(stream)))
    return out


def mla_decode(q, kv_latent, k_pe, W_kvb, W_o, W_kvb_scale=None, W_o_scale=None, topk_idx=None,
               scale=192 ** -0.5, out=None, workspace=None, stream=None):
    """One new position per sequence against its cache: q [B,H,192], kv_latent [B,T,512], k_pe [B,T,64]
    (the new position's cache row last), topk_idx int32 [B, topk] or None -> out bf16 [B, 7168]."""
    B, H, _ = q.shape
    T = kv_latent.shape[1]
    topk = 0 if topk_idx is None else topk_idx.shape[-1]
    fp8 = _wtype(W_kvb)
    if _wtype(W_o) != fp8:
        raise ValueError("W_kvb and W_o must use the same storage type")
    if topk_idx is not None and topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32")
    dims = make_dims(B, T, H, topk, fp8)
    if out is None:
        out = _new((B, D_MODEL), torch.bfloat16, q.device, stream)
    ws, nbytes = _workspace(dims, MLA_ENTRY_DECODE, topk_idx is not None, workspace, q.device, stream)
    lib = load_library()
    _check("mla_decode", lib.mla_decode(ctypes.byref(dims), _ptr(q), _ptr(kv_latent), _ptr(k_pe), _ptr(W_kvb),
                                        _ptr(W_kvb_scale), _ptr(W_o), _ptr(W_o_scale), _ptr(topk_idx), float(scale),
                                        _ptr(out), _ptr(ws), nbytes, _stream(stream)))
    return out


def mla_quantize_act(x, codes=None, scales=None, stream=None):
    """Dynamic e4m3 quantization of x bf16 [rows, cols] (cols % 128 == 0) ->
    (codes uint8 [rows, cols], scales float32 [cols // 128, rows]), s = amax / 448 per group."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    rows, cols = x.reshape(-1, x.shape[-1]).shape
    if codes is None:
        codes = _new((rows, cols), torch.uint8, x.device, stream)
    if scales is None:
        scales = _new((cols // 128 if cols % 128 == 0 else 0, rows), torch.float32, x.device, stream)
    _check("mla_quantize_act", load_library().mla_quantize_act(_ptr(x), rows, cols, _ptr(codes), _ptr(scales),
                                                               _stream(stream)))
    return codes, scales


# ------------------------------------------------------------------ serving over a paged cache


# These calls take two microseconds on the device at the smallest sizes, so their host side is kept short: tensors are
# asked for few attributes, and for none twice.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream's handle without its object
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_BF16, _I32 = torch.bfloat16, torch.int32


def _expect(t, name, dtype, shape=None):
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


def _cuda(t):
    """Index of the tensor's CUDA device."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensor must be on a CUDA device")
    return index


def _data(t, index, strided=False):
    """Address of a tensor that has to be on CUDA device `index` and, unless `strided`, contiguous; None for None."""
    if t is None:
        return None
    if t.get_device() != index:
        raise ValueError(f"the tensors are on cuda:{index} and {t.device}")
    if not (strided or t.is_contiguous()):
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _call(name, index, stream, args):
    """Runs an entry point on CUDA device `index`, on `stream` or that device's current stream."""
    fn = getattr(_lib or load_library(), name)
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{index}")
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(index)
    else:
        handle = torch.cuda.current_stream(index).cuda_stream
    if index == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != 0:
        raise MlaError(name, rc)


def make_rope(base=10000.0, layout=MLA_ROPE_INTERLEAVED, scaling=MLA_ROPE_UNSCALED, factor=1.0, original_len=4096,
              beta_fast=32.0, beta_slow=1.0, magnitude=1.0) -> MlaRopeTable:
    """Rotary settings of a model (the frequencies of the 32 pairs, scaled for long contexts), made once and
    passed to mla_rope and mla_cache_append."""
    table = MlaRopeTable()
    _check("mla_rope_init", load_library().mla_rope_init(
        ctypes.byref(table), int(layout), float(base), int(scaling), float(factor), float(original_len),
        float(beta_fast), float(beta_slow), float(magnitude)))
    return table


def _rows_and_heads(t, shape, lead):
    """(rows, row stride, heads, head stride) of a tensor [*lead, H, W] or [*lead, W] whose last dimension is
    contiguous and whose leading ones fold into one."""
    n = len(shape)
    if n != lead + 1 and n != lead + 2:
        raise ValueError("the tensor must be [*positions.shape, heads, width] or [*positions.shape, width]")
    width = shape[-1]
    heads = shape[-2] if n == lead + 2 else 1
    if t.is_contiguous():
        row = heads * width
        return (t.numel() // row if row else 0), row, heads, width
    strides = t.stride()
    if strides[-1] != 1:
        raise ValueError("the tensor's last dimension must be contiguous")
    rows, row = 1, 0
    for d in reversed(range(lead)):
        if shape[d] == 1:
            continue
        if rows == 1:
            row = strides[d]
        elif strides[d] != row * rows:
            raise ValueError("the leading dimensions must fold into one")
        rows *= shape[d]
    return rows, row, heads, strides[-2] if heads > 1 else width


def mla_rope(x, positions, rope, offset=None, out=None, inverse=False, stream=None):
    """Rotates 64 elements of every head by its token's position: x bf16 [*positions.shape, H, W] (or without H),
    positions int32; elements [offset, offset + 64) (default: the last 64) are turned, the others copied. `out` may be
    x (in place). Strided x and out are taken as they are. inverse=True rotates back (the transposed map: with
    x = d out, the gradient). `rope` comes from make_rope."""
    if not (x.dtype is _BF16 and positions.dtype is _I32):
        raise ValueError("x must be torch.bfloat16 and positions torch.int32")
    shape, at = x.shape, positions.shape
    lead = len(at)
    rows, x_row, heads, x_head = _rows_and_heads(x, shape, lead)
    if shape[:lead] != at:
        raise ValueError(f"x {tuple(shape)} does not start with the shape of positions {tuple(at)}")
    index = _cuda(x)
    if out is None:
        out = _new(shape, _BF16, x.device, stream)
    if out is x:
        o_row, o_head = x_row, x_head
    else:
        _expect(out, "out", _BF16, shape)
        _, o_row, _, o_head = _rows_and_heads(out, shape, lead)
    width = shape[-1]
    _call("mla_rope", index, stream,
          (ctypes.byref(rope), x.data_ptr(), x_row, x_head, _data(out, index, True), o_row, o_head, rows, heads, width,
           width - D_ROPE if offset is None else int(offset), _data(positions, index), 1 if inverse else 0))
    return out


def mla_cache_append(kv_a, norm_weight, positions, rope, kv_cache, k_pe_cache, slots=None, eps=1e-6, stream=None):
    """Latent RMSNorm and key rotation in one pass, into cache rows: kv_a bf16 [*positions.shape, 576] (rows may be
    strided), norm_weight bf16 or float32 [512], positions int32; slots int32, one cache row per token (-1: skip), or
    None: token r to row r. kv_cache bf16 [..., 512] and k_pe_cache bf16 [..., 64] are contiguous with the same number
    of rows (pages [P, page, 512], or mla_prefill's kv_latent [B, T, 512]). Returns (kv_cache, k_pe_cache)."""
    if not (kv_a.dtype is kv_cache.dtype is k_pe_cache.dtype is _BF16 and positions.dtype is _I32):
        raise ValueError("kv_a, kv_cache and k_pe_cache must be torch.bfloat16 and positions torch.int32")
    f32 = norm_weight.dtype is torch.float32
    if not (f32 or norm_weight.dtype is _BF16) or norm_weight.shape != (D_LATENT,):
        raise ValueError("norm_weight must be bf16 or float32 [512]")
    shape, at = kv_a.shape, positions.shape
    if shape != (*at, D_LATENT + D_ROPE):
        raise ValueError("kv_a must be [*positions.shape, 576]")
    rows, stride, _, _ = _rows_and_heads(kv_a, shape, len(at))
    if rows <= 1:
        stride = D_LATENT + D_ROPE
    if slots is not None:
        _expect(slots, "slots", _I32, at)
    latent = kv_cache.shape
    if latent[-1] != D_LATENT or k_pe_cache.shape != (*latent[:-1], D_ROPE):
        raise ValueError("kv_cache must be [..., 512] and k_pe_cache [..., 64] over the same rows")
    cache_rows = kv_cache.numel() // D_LATENT
    if slots is None and cache_rows < rows:
        raise ValueError("the cache has fewer rows than there are tokens")
    index = _cuda(kv_a)
    _call("mla_cache_append", index, stream,
          (ctypes.byref(rope), kv_a.data_ptr(), stride, _data(norm_weight, index), 1 if f32 else 0, float(eps),
           _data(positions, index), _data(slots, index), rows, _data(kv_cache, index), _data(k_pe_cache, index),
           cache_rows))
    return kv_cache, k_pe_cache


def _pages(kv_cache, k_pe_cache, table_width, one_layer):
    if not kv_cache.dtype is k_pe_cache.dtype is _BF16:
        raise ValueError("kv_cache and k_pe_cache must be torch.bfloat16")
    shape = kv_cache.shape
    n = len(shape)
    if (n != 3 and (one_layer or n != 4)) or shape[-1] != D_LATENT:
        raise ValueError("kv_cache must be [pages, page_size, 512]" +
                         ("" if one_layer else " or [layers, pages, page_size, 512]"))
    if k_pe_cache.shape != (*shape[:-1], D_ROPE):
        raise ValueError("k_pe_cache must be [..., 64] over kv_cache's pages")
    return MlaPages(shape[-3], shape[-2], table_width, shape[0] if n == 4 else 1)


def mla_tree_decode(q, kv_cache, k_pe_cache, block_table, cache_len, W_kvb, W_o, W_kvb_scale=None, W_o_scale=None,
                    parents=None, n_nodes=None, scale=192 ** -0.5, out=None, workspace=None, stream=None):
    """Attention of up to 64 new tokens per sequence over a paged cache, and W_o: q bf16 [B, N, H, 192], kv_cache
    [pages, page_size, 512], k_pe_cache [pages, page_size, 64], block_table int32 [B, width], cache_len int32 [B]
    (committed positions; node j of a sequence is cached at position cache_len + j), n_nodes int32 [B] or None (all N),
    parents int32 [B, N] (the node each hangs below, -1: the last committed position) or None: a chain
    -> out bf16 [B, N, 7168], 0 for nodes from n_nodes on."""
    _expect(q, "q", torch.bfloat16)
    if q.dim() != 4 or q.shape[-1] != D_NOPE + D_ROPE:
        raise ValueError("q must be [B, N, H, 192]")
    B, N, H, _ = q.shape
    _expect(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, width]")
    _expect(cache_len, "cache_len", torch.int32, (B,))
    if n_nodes is not None:
        _expect(n_nodes, "n_nodes", torch.int32, (B,))
    if parents is not None:
        _expect(parents, "parents", torch.int32, (B, N))
    fp8 = _wtype(W_kvb)
    if _wtype(W_o) != fp8:
        raise ValueError("W_kvb and W_o must use the same storage type")
    if W_kvb.shape != (H * (D_NOPE + D_V), D_LATENT) or W_o.shape != (H * D_V, D_MODEL):
        raise ValueError("W_kvb must be [H*256, 512] and W_o [H*128, 7168]")
    if fp8:
        for w, s, name in ((W_kvb, W_kvb_scale, "W_kvb_scale"), (W_o, W_o_scale, "W_o_scale")):
            if s is None:
                raise ValueError(f"e4m3 weights need {name}")
            _expect(s, name, torch.float32, (w.shape[0] // 128, w.shape[1] // 128))
    pages = _pages(kv_cache, k_pe_cache, block_table.shape[1], True)
    index = _cuda(q)
    dims = make_dims(B, N, H, 0, fp8)
    if out is None:
        out = _new((B, N, D_MODEL), torch.bfloat16, q.device, stream)
    else:
        _expect(out, "out", torch.bfloat16, (B, N, D_MODEL))
    ws, nbytes = _workspace(dims, MLA_ENTRY_TREE_DECODE, False, workspace, q.device, stream)
    _call("mla_tree_decode", index, stream,
          (ctypes.byref(dims), ctypes.byref(pages), _data(q, index), _data(kv_cache, index), _data(k_pe_cache, index),
           _data(block_table, index), _data(cache_len, index), _data(n_nodes, index), _data(parents, index),
           _data(W_kvb, index), _data(W_kvb_scale, index), _data(W_o, index), _data(W_o_scale, index), float(scale),
           _data(out, index), _data(ws, index), nbytes))
    return out


def mla_cache_compact(kv_cache, k_pe_cache, block_table, cache_len, accepted, n_accepted, stream=None):
    """Moves each sequence's accepted rows together: position cache_len + accepted[b, i] to cache_len + i for
    i < n_accepted[b], in every layer. kv_cache [pages, page_size, 512] or [layers, pages, page_size, 512] (k_pe_cache
    alike with 64), accepted int32 [B, width <= 64], the others int32 [B]."""
    if not (block_table.dtype is accepted.dtype is cache_len.dtype is n_accepted.dtype is _I32):
        raise ValueError("block_table, cache_len, accepted and n_accepted must be torch.int32")
    table, nodes = block_table.shape, accepted.shape
    if len(table) != 2 or len(nodes) != 2 or table[0] != nodes[0]:
        raise ValueError("block_table and accepted must be [B, width]")
    B = table[0]
    if not cache_len.shape == n_accepted.shape == (B,):
        raise ValueError("cache_len and n_accepted must be [B]")
    pages = _pages(kv_cache, k_pe_cache, table[1], False)
    index = _cuda(kv_cache)
    _call("mla_cache_compact", index, stream,
          (ctypes.byref(pages), _data(kv_cache, index), _data(k_pe_cache, index), _data(block_table, index),
           _data(cache_len, index), _data(accepted, index), _data(n_accepted, index), B, nodes[1]))


def mla_cache_copy_pages(kv_cache, k_pe_cache, src, dst, stream=None):
    """Copies page src[i] onto page dst[i] in every layer. src and dst are host lists (sequences of ints or int32 CPU
    tensors) of equal length; a destination may be listed once and be no other pair's source. The caches are as for
    mla_cache_compact."""
    lists = []
    for v in (src, dst):
        if isinstance(v, torch.Tensor):
            if v.is_cuda:
                raise ValueError("src and dst are host lists, not CUDA tensors")
            v = v.tolist()
        elif isinstance(v, (bytes, bytearray)):  # array takes these as raw memory, four to an index
            raise ValueError("src and dst are sequences of ints")
        lists.append(array.array("i", v))  # OverflowError for an index beyond 32 bits
    n = len(lists[0])  # of what the call reads
    if len(lists[1]) != n:
        raise ValueError("src and dst must have the same length")
    pages = _pages(kv_cache, k_pe_cache, 0, False)
    index = _cuda(kv_cache)
    _call("mla_cache_copy_pages", index, stream,
          (ctypes.byref(pages), _data(kv_cache, index), _data(k_pe_cache, index), lists[0].buffer_info()[0],
           lists[1].buffer_info()[0], n))


def mla_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error word."""
    v = ctypes.c_int(0)
    _check("mla_device_status", load_library().mla_device_status(_stream(stream), ctypes.byref(v)))
    return v.value


def mla_set_e4m3_weight_conversion(onchip: bool):
    """e4m3 weights with bf16 activations: False (default) dequantises them
    into a bf16 workspace copy per call; True converts them on chip inside
    the projection GEMMs (bit-identical, no copy). Query workspace sizes
    after switching."""
    _check("mla_set_e4m3_weight_conversion", load_library().mla_set_e4m3_weight_conversion(1 if onchip else 0))


def mla_set_wait_timeout_ns(ns: int):
    """Time limit of the kernels' on-chip waits on the current device, for
    launches from now on (0 restores the 1 s default)."""
    _check("mla_set_wait_timeout_ns", load_library().mla_set_wait_timeout_ns(int(ns)))


def mla_test_withhold_attention_loads(on):
    """Test hook: while on, a kernel's producer stops issuing loads and its
    bounded waits expire (error word 1xx, clean exit). True or 1: block-dense
    attention; 2: tree attention, after a tile's first block; 3: few-row
    GEMMs, after a CTA's first tile. False or 0: off."""
    _check("mla_test_withhold_attention_loads", load_library().mla_test_withhold_attention_loads(int(on)))


def mla_profile_begin():
    _check("mla_profile_begin", load_library().mla_profile_begin())


def mla_profile_end():
    """{class name: (total ms, launches)} for the launches since mla_profile_begin()."""
    ms = (ctypes.c_float * MLA_PROFILE_CLASSES)()
    n = (ctypes.c_int * MLA_PROFILE_CLASSES)()
    _check("mla_profile_end", load_library().mla_profile_end(ms, n))
    return {PROFILE_CLASS_NAMES[i]: (float(ms[i]), int(n[i])) for i in range(MLA_PROFILE_CLASSES)}


class PrefillPipeline:
    """mla_prefill over a stream of host batches, with the copies overlapped.

    For batch i the host inputs (pinned CPU tensors) are copied to the device
    on a copy stream while the kernels of batch i-1 run on the compute stream
    and the output of batch i-2 is copied back on a third stream. Two device
    buffer sets alternate; the weights stay resident. Every kernel is the C
    ABI's; this class only orders copies and launches with CUDA events.
    """

    _INPUTS = ("q", "kv_latent", "k_pe", "topk_idx")

    def __init__(self, B, T, H, W_kvb, W_o, W_kvb_scale=None, W_o_scale=None, topk=None,
                 scale=192 ** -0.5, device=None, path=MLA_PATH_AUTO, act=MLA_ACT_BF16):
        dev = torch.device(device) if device is not None else W_o.device
        self.dev, self.scale = dev, float(scale)
        self.w = dict(W_kvb=W_kvb, W_o=W_o, W_kvb_scale=W_kvb_scale, W_o_scale=W_o_scale)
        shapes = {"q": ((B, T, H, D_NOPE + D_ROPE), torch.bfloat16), "kv_latent": ((B, T, D_LATENT), torch.bfloat16),
                  "k_pe": ((B, T, D_ROPE), torch.bfloat16)}
        if topk is not None:
            shapes["topk_idx"] = ((B, T, int(topk)), torch.int32)
        self.slots = [{k: torch.empty(s, dtype=d, device=dev) for k, (s, d) in shapes.items()} for _ in range(2)]
        for sl in self.slots:
            sl["out"] = torch.empty(B, T, D_MODEL, dtype=torch.bfloat16, device=dev)
        self.act, self.path = int(act), int(path)
        dims = make_dims(B, T, H, 0 if topk is None else topk, _wtype(W_kvb), path=self.path, act=self.act)
        self.ws = torch.empty(max(1, mla_workspace_bytes(dims, MLA_ENTRY_PREFILL, topk is not None)),
                              dtype=torch.uint8, device=dev)
        self.h2d, self.comp, self.d2h = (torch.cuda.Stream(dev) for _ in range(3))
        # The buffers are the current stream's: its work on what the blocks held before comes first, and they are not
        # handed out again before the three streams are done with them.
        for st in (self.h2d, self.comp, self.d2h):
            st.wait_stream(torch.cuda.current_stream(dev))
            for t in (self.ws, *(t for sl in self.slots for t in sl.values())):
                t.record_stream(st)
        ev = lambda: [torch.cuda.Event() for _ in range(2)]  # noqa: E731
        self.ev_in, self.ev_done, self.ev_out = ev(), ev(), ev()
        self.used = [False, False]
        self.i = 0

    def submit(self, host_inputs: dict, host_out: torch.Tensor):
        """Queues one batch: host_inputs maps q, kv_latent, k_pe (and topk_idx)
        to pinned CPU tensors; the result lands in the pinned host_out."""
        k = self.i & 1
        sl = self.slots[k]
        with torch.cuda.stream(self.h2d):
            if self.used[k]:
                self.h2d.wait_event(self.ev_done[k])  # the kernels that read this slot are done
            for name in self._INPUTS:
                if name in sl:
                    sl[name].copy_(host_inputs[name], non_blocking=True)
            self.ev_in[k].record(self.h2d)
        self.comp.wait_event(self.ev_in[k])
        if self.used[k]:
            self.comp.wait_event(self.ev_out[k])  # the previous output of this slot has been copied out
        mla_prefill(sl["q"], sl["kv_latent"], sl["k_pe"], self.w["W_kvb"], self.w["W_o"], self.w["W_kvb_scale"],
                    self.w["W_o_scale"], topk_idx=sl.get("topk_idx"), scale=self.scale, out=sl["out"],
                    workspace=self.ws, stream=self.comp, path=self.path, act=self.act)
        self.ev_done[k].record(self.comp)
        with torch.cuda.stream(self.d2h):
            self.d2h.wait_event(self.ev_done[k])
            host_out.copy_(sl["out"], non_blocking=True)
            self.ev_out[k].record(self.d2h)
        self.used[k] = True
        self.i += 1

    def synchronize(self):
        for s in (self.h2d, self.comp, self.d2h):
            s.synchronize()
