"""ctypes binding of libpagedattn.so: the C ABI under the same names.

This layer only marshals arguments: torch tensors become raw pointers, the
stream defaults to torch's current CUDA stream, and a non-zero status raises
``PagedAttnError``.  Every step of the attention path runs in the library's
CUDA kernels; there is no fallback.  If the shared library has not been built
the first call fails loudly with instructions.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpagedattn.so")

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_ARCH = 0, 1, 2, 3
PA_ERR_WORKSPACE, PA_ERR_CUDA, PA_ERR_DEVICE_INDEX = 4, 5, 6
PA_MODE_DECODE, PA_MODE_EXTEND, PA_MODE_SAGE_DECODE, PA_MODE_SAGE_SPARSE, PA_MODE_TREE = 0, 1, 2, 3, 4

EXPORTED = ("pa_plan_workspace_size", "attn_plan", "attn_decode_paged", "attn_extend_paged",
            "attn_decode_paged_sage", "attn_debug_gather", "pa_read_device_error",
            "pa_status_string", "pa_version", "attn_decode_paged_noalloc", "attn_kv_store",
            "attn_kv_store_sage", "attn_decode_paged_fp8", "attn_plan_sage_sparse", "attn_extend_paged_sage",
            "pa_noalloc_read_device_error", "attn_plan_tree", "attn_tree_paged", "attn_tree_paged_fp8",
            "attn_tree_verify", "attn_kv_compact")


class pa_plan_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "mode", "batch", "hq", "hkv", "head_dim", "page_size", "max_kv_len", "max_q_tokens",
        "num_sms", "max_splits", "sage_k_block", "reserved")]


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


_lib = None
_P = ctypes.c_void_p
_I32, _I64, _F32, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load (once) and return the shared library; raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m paged_kv_flashattention_split_b200.build` "
                "(or __graft_entry__.build()).  There is no CPU fallback.")
        L = ctypes.CDLL(LIB_PATH)
        PP = ctypes.POINTER(pa_plan_params)
        sig = {
            "pa_plan_workspace_size": (_I32, [PP, ctypes.POINTER(_SZ)]),
            "attn_plan": (_I32, [PP, _P, _P, _P, _SZ, _P]),
            "attn_plan_sage_sparse": (_I32, [PP, _P, _P, _I64, _P, _SZ, _P]),
            "attn_decode_paged": (_I32, [PP, _P, _SZ, _P, _P, _P, _I64, _P, _I64, _F32, _P, _P, _P]),
            "attn_extend_paged": (_I32, [PP, _P, _SZ, _P, _P, _P, _I64, _P, _I64, _F32, _P, _P, _P]),
            "attn_decode_paged_fp8": (_I32, [PP, _P, _SZ, _P, _P, _P, _F32, _F32, _I64, _P, _I64, _F32, _P, _P,
                                             _P]),
            "attn_decode_paged_sage": (_I32, [PP, _P, _SZ, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64,
                                              _P, _P]),
            "attn_extend_paged_sage": (_I32, [PP, _P, _SZ, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _I64, _P, _P]),
            "attn_debug_gather": (_I32, [_P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P, _I64,
                                         _P, _P, _P]),
            "pa_read_device_error": (_I32, [_P, _P]),
            "pa_noalloc_read_device_error": (_I32, [_P]),
            "attn_kv_store": (_I32, [_P, _P, _P, _I64, _I32, _I32, _P, _P, _I64, _P, _P]),
            "attn_kv_store_sage": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _P, _P, _P, _I64, _P, _P]),
            "attn_decode_paged_noalloc": (_I32, [PP, _P, _P, _P, _P, _I64, _P, _I64, _F32, _P, _P, _P]),
            "attn_plan_tree": (_I32, [PP, _P, _P, _P, _P, _SZ, _P]),
            "attn_tree_paged": (_I32, [PP, _P, _SZ, _P, _P, _P, _I64, _P, _I64, _F32, _P, _P, _P]),
            "attn_tree_paged_fp8": (_I32, [PP, _P, _SZ, _P, _P, _P, _F32, _F32, _I64, _P, _I64, _F32, _P, _P, _P]),
            "attn_tree_verify": (_I32, [_I32, _I32, _I32, _P, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P,
                                        _P, _P]),
            "attn_kv_compact": (_I32, [ctypes.POINTER(_P), _I32, _I32, _I32, _I32, _I64, _I32, _I32, _P, _P, _P, _P,
                                       _I64, _P, _I64, _I32, _P, _P, _P]),
            "pa_status_string": (ctypes.c_char_p, [_I32]),
            "pa_version": (_I32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pa_status_string(int(status)).decode()


def _ptr(t):
    """Device (or host) address of a tensor, an int address, or None -> NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without the Stream object around it, and whether there is a device at all without
# asking the driver again (a fifth and a twentieth of a small call's host time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_initialised = torch.cuda.is_initialized


def _stream(stream):
    if stream is None:
        if not _initialised() and not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str, raise_on_error: bool):
    if raise_on_error and status != PA_OK:
        raise PagedAttnError(status, where)
    return status


def make_params(mode: int, batch: int, hq: int, hkv: int, head_dim: int = 128, page_size: int = 1,
                max_kv_len: int = 0, max_q_tokens: int = 0, num_sms: int = 0, max_splits: int = 0,
                sage_k_block: int = 0) -> pa_plan_params:
    return pa_plan_params(mode, batch, hq, hkv, head_dim, page_size, max_kv_len, max_q_tokens,
                          num_sms, max_splits, sage_k_block, 0)


def pa_plan_workspace_size(params: pa_plan_params, raise_on_error: bool = True):
    out = _SZ(0)
    st = lib().pa_plan_workspace_size(ctypes.byref(params), ctypes.byref(out))
    _check(st, "pa_plan_workspace_size", raise_on_error)
    return out.value if st == PA_OK else st


def attn_plan(params, seq_lens, cu_seqlens_q, ws, stream=None, raise_on_error=True) -> int:
    nbytes = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    st = lib().attn_plan(ctypes.byref(params), _ptr(seq_lens), _ptr(cu_seqlens_q), _ptr(ws), nbytes,
                         _stream(stream))
    return _check(st, "attn_plan", raise_on_error)


def attn_plan_sage_sparse(params, seq_lens, block_mask, ws, stream=None, raise_on_error=True) -> int:
    """Plan of the block-sparse Sage decode; block_mask uint8 [B, mask_pitch] (nonzero = attend)."""
    nbytes = ws.numel() * ws.element_size() if isinstance(ws, torch.Tensor) else 0
    st = lib().attn_plan_sage_sparse(ctypes.byref(params), _ptr(seq_lens), _ptr(block_mask),
                                     int(block_mask.shape[-1]), _ptr(ws), nbytes, _stream(stream))
    return _check(st, "attn_plan_sage_sparse", raise_on_error)


def attn_decode_paged(params, ws, q, k_pool, v_pool, page_table, sm_scale, out, lse_out=None,
                      num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    num_slots = k_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_decode_paged(ctypes.byref(params), _ptr(ws), ws.numel() * ws.element_size(),
                                 _ptr(q), _ptr(k_pool), _ptr(v_pool), int(num_slots), _ptr(page_table),
                                 int(pt_pitch), float(sm_scale), _ptr(out), _ptr(lse_out),
                                 _stream(stream))
    return _check(st, "attn_decode_paged", raise_on_error)


def attn_decode_paged_fp8(params, ws, q, k8_pool, v8_pool, k_scale, v_scale, page_table, sm_scale, out,
                          lse_out=None, num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    """DECODE over E4M3 pools (uint8 codes) dequantised by k_scale / v_scale; q and out bf16."""
    num_slots = k8_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_decode_paged_fp8(ctypes.byref(params), _ptr(ws), ws.numel() * ws.element_size(),
                                     _ptr(q), _ptr(k8_pool), _ptr(v8_pool), float(k_scale), float(v_scale),
                                     int(num_slots), _ptr(page_table), int(pt_pitch), float(sm_scale), _ptr(out),
                                     _ptr(lse_out), _stream(stream))
    return _check(st, "attn_decode_paged_fp8", raise_on_error)


def attn_extend_paged(params, ws, q, k_pool, v_pool, page_table, sm_scale, out, lse_out=None,
                      num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    num_slots = k_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_extend_paged(ctypes.byref(params), _ptr(ws), ws.numel() * ws.element_size(),
                                 _ptr(q), _ptr(k_pool), _ptr(v_pool), int(num_slots), _ptr(page_table),
                                 int(pt_pitch), float(sm_scale), _ptr(out), _ptr(lse_out),
                                 _stream(stream))
    return _check(st, "attn_extend_paged", raise_on_error)


def attn_decode_paged_sage(params, ws, q8, sf_q, k8_pool, v8_pool, sf_k, sf_v, v_mean, page_table,
                           out, num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    num_slots = k8_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_decode_paged_sage(ctypes.byref(params), _ptr(ws), ws.numel() * ws.element_size(),
                                      _ptr(q8), _ptr(sf_q), _ptr(k8_pool), _ptr(v8_pool), _ptr(sf_k),
                                      _ptr(sf_v), _ptr(v_mean), int(num_slots), _ptr(page_table),
                                      int(pt_pitch), _ptr(out), _stream(stream))
    return _check(st, "attn_decode_paged_sage", raise_on_error)


def attn_extend_paged_sage(params, ws, q8, sf_q, k8_pool, v8_pool, sf_k, sf_v, v_mean, page_table, out,
                           num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    """8-bit Sage EXTEND over an EXTEND plan with page size 64; q8 int8 [T, Hq, D], out bf16."""
    num_slots = k8_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_extend_paged_sage(ctypes.byref(params), _ptr(ws), ws.numel() * ws.element_size(),
                                      _ptr(q8), _ptr(sf_q), _ptr(k8_pool), _ptr(v8_pool), _ptr(sf_k),
                                      _ptr(sf_v), _ptr(v_mean), int(num_slots), _ptr(page_table),
                                      int(pt_pitch), _ptr(out), _stream(stream))
    return _check(st, "attn_extend_paged_sage", raise_on_error)


def attn_debug_gather(seq_lens, r, h_kv, hkv, page_size, max_len, k_pool, page_table, slots_out,
                      rows_out, head_dim=128, num_slots=None, pt_pitch=None, stream=None,
                      raise_on_error=True) -> int:
    num_slots = k_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_debug_gather(_ptr(seq_lens), r, h_kv, hkv, head_dim, page_size, max_len,
                                 _ptr(k_pool), int(num_slots), _ptr(page_table), int(pt_pitch),
                                 _ptr(slots_out), _ptr(rows_out), _stream(stream))
    return _check(st, "attn_debug_gather", raise_on_error)


def attn_decode_paged_noalloc(params, seq_lens, q, k_pool, v_pool, page_table, sm_scale, out, lse_out=None,
                              num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    """Plan and decode without a caller workspace (the library's fixed 16 MiB array is used)."""
    num_slots = k_pool.shape[0] if num_slots is None else num_slots
    pt_pitch = page_table.shape[-1] if pt_pitch is None else pt_pitch
    st = lib().attn_decode_paged_noalloc(ctypes.byref(params), _ptr(seq_lens), _ptr(q), _ptr(k_pool),
                                         _ptr(v_pool), int(num_slots), _ptr(page_table), int(pt_pitch),
                                         float(sm_scale), _ptr(out), _ptr(lse_out), _stream(stream))
    return _check(st, "attn_decode_paged_noalloc", raise_on_error)


def attn_kv_store(k_new, v_new, out_cache_loc, k_pool, v_pool, ws=None, n_tokens=None, num_slots=None,
                  stream=None, raise_on_error=True) -> int:
    """Scatter new tokens' K/V rows ([n, Hkv, D] bf16) into the pools at out_cache_loc (int32 [n])."""
    n = k_new.shape[0] if n_tokens is None else n_tokens
    num_slots = k_pool.shape[0] if num_slots is None else num_slots
    hkv = k_pool.shape[1]
    st = lib().attn_kv_store(_ptr(k_new), _ptr(v_new), _ptr(out_cache_loc), int(n), int(hkv), int(k_pool.shape[2]),
                             _ptr(k_pool), _ptr(v_pool), int(num_slots), _ptr(ws), _stream(stream))
    return _check(st, "attn_kv_store", raise_on_error)


def attn_kv_store_sage(k8_new, v8_new, sf_k_new, out_cache_loc, k8_pool, v8_pool, sf_k, ws=None, n_tokens=None,
                       num_slots=None, stream=None, raise_on_error=True) -> int:
    """Scatter new tokens' K8/V8 rows ([n, Hkv, D] bytes) into the 8-bit pools, and the block
    scales sf_k_new ([n, Hkv] fp32, or None) of the tokens that open a 64-slot block."""
    n = k8_new.shape[0] if n_tokens is None else n_tokens
    num_slots = k8_pool.shape[0] if num_slots is None else num_slots
    hkv = k8_pool.shape[1]
    st = lib().attn_kv_store_sage(_ptr(k8_new), _ptr(v8_new), _ptr(sf_k_new), _ptr(out_cache_loc), int(n), int(hkv),
                                  int(k8_pool.shape[2]), _ptr(k8_pool), _ptr(v8_pool), _ptr(sf_k), int(num_slots),
                                  _ptr(ws), _stream(stream))
    return _check(st, "attn_kv_store_sage", raise_on_error)


_Tensor, _int32, _float32 = torch.Tensor, torch.int32, torch.float32


def _here() -> int:
    """Index of the current device, -1 without one (as a host tensor's get_device)."""
    if _initialised() or torch.cuda.is_available():
        return torch.cuda.current_device()
    return -1


def _stream_of(here, stream):
    """The stream's handle; the current one of the current device if none is given."""
    if stream is None and _raw_stream is not None and here >= 0:
        return _raw_stream(here)
    return _stream(stream)


def _elsewhere(name, t):
    """A tensor that is not on the current device: pinned host memory is within its reach, all else would fault."""
    if t.device.type != "cpu" or not t.is_pinned():
        raise ValueError(f"{name}: on {t.device}, not on the current device")


def _vector(name, t, dtype, here, n=0):
    """Address of a dense tensor of at least n values of one type on device `here`; an int is an address, None is NULL.
    The kernels read 32-bit words: 64-bit tokens, as argmax and topk give them, would be taken for other tokens."""
    if type(t) is not _Tensor and (t is None or isinstance(t, int)):
        return t
    if t.dtype is not dtype or (n and t.numel() < n) or not t.is_contiguous():
        raise ValueError(f"{name}: a dense {dtype} tensor of at least {n} values is needed")
    if t.get_device() != here:
        _elsewhere(name, t)
    return t.data_ptr()


def _workspace(ws, here):
    """Address of a plan workspace."""
    if type(ws) is not _Tensor and (ws is None or isinstance(ws, int)):
        return ws
    if not ws.is_contiguous():
        raise ValueError("ws: a dense tensor is needed")
    if ws.get_device() != here:
        _elsewhere("ws", ws)
    return ws.data_ptr()


_BITS16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))          # bf16, or its bit patterns
_BITS8 = frozenset((torch.uint8, torch.int8, torch.float8_e4m3fn))        # E4M3 codes


def _dense(name, t, kinds, here):
    """Address of a dense tensor of one of the given types on device `here` (an int is an address, None is NULL)."""
    if type(t) is not _Tensor and (t is None or isinstance(t, int)):
        return t
    if t.dtype not in kinds or not t.is_contiguous():
        raise ValueError(f"{name}: a dense tensor of one of {sorted(map(str, kinds))} is needed")
    if t.get_device() != here:
        _elsewhere(name, t)
    return t.data_ptr()


def _table(page_table, batch, pt_pitch, here):
    """Address and pitch of a page table: dense, or columns of longer rows with their pitch given."""
    if pt_pitch is None:
        pt_pitch = page_table.shape[-1]
        return _vector("page_table", page_table, _int32, here, batch * pt_pitch), int(pt_pitch)
    if isinstance(page_table, _Tensor):
        if page_table.dtype is not _int32:
            raise ValueError("page_table: int32 is needed")
        if page_table.get_device() != here:
            _elsewhere("page_table", page_table)
    return _ptr(page_table), int(pt_pitch)


def attn_plan_tree(params, seq_lens, cu_seqlens_q, parent, ws, stream=None, raise_on_error=True) -> int:
    """Plan of the draft-tree attention; parent int32 [sum n] (-1 a root, -2 a node not in use)."""
    batch, here = params.batch, _here()
    st = lib().attn_plan_tree(ctypes.byref(params), _vector("seq_lens", seq_lens, _int32, here, batch),
                              _vector("cu_seqlens_q", cu_seqlens_q, _int32, here, batch + 1),
                              _vector("parent", parent, _int32, here), _workspace(ws, here),
                              ws.numel() * ws.element_size(), _stream_of(here, stream))
    return _check(st, "attn_plan_tree", raise_on_error)


def attn_tree_paged(params, ws, q, k_pool, v_pool, page_table, sm_scale, out, lse_out=None, num_slots=None,
                    pt_pitch=None, stream=None, raise_on_error=True) -> int:
    """Draft-tree attention for one layer over a TREE plan; q and out bf16 [sum n, Hq, D]."""
    num_slots = k_pool.shape[0] if num_slots is None else num_slots
    here = _here()
    table, pt_pitch = _table(page_table, params.batch, pt_pitch, here)
    st = lib().attn_tree_paged(ctypes.byref(params), _workspace(ws, here), ws.numel() * ws.element_size(),
                               _dense("q", q, _BITS16, here), _dense("k_pool", k_pool, _BITS16, here),
                               _dense("v_pool", v_pool, _BITS16, here), int(num_slots), table, pt_pitch,
                               float(sm_scale), _dense("out", out, _BITS16, here),
                               _vector("lse_out", lse_out, _float32, here), _stream_of(here, stream))
    return _check(st, "attn_tree_paged", raise_on_error)


def attn_tree_paged_fp8(params, ws, q, k8_pool, v8_pool, k_scale, v_scale, page_table, sm_scale, out, lse_out=None,
                        num_slots=None, pt_pitch=None, stream=None, raise_on_error=True) -> int:
    """Draft-tree attention over E4M3 pools (uint8 codes) dequantised by k_scale / v_scale; q and out bf16."""
    num_slots = k8_pool.shape[0] if num_slots is None else num_slots
    here = _here()
    table, pt_pitch = _table(page_table, params.batch, pt_pitch, here)
    st = lib().attn_tree_paged_fp8(ctypes.byref(params), _workspace(ws, here), ws.numel() * ws.element_size(),
                                   _dense("q", q, _BITS16, here), _dense("k8_pool", k8_pool, _BITS8, here),
                                   _dense("v8_pool", v8_pool, _BITS8, here), float(k_scale), float(v_scale),
                                   int(num_slots), table, pt_pitch, float(sm_scale),
                                   _dense("out", out, _BITS16, here), _vector("lse_out", lse_out, _float32, here),
                                   _stream_of(here, stream))
    return _check(st, "attn_tree_paged_fp8", raise_on_error)


def attn_tree_verify(cu_seqlens_q, parent, tokens, target_probs, draft_probs, u_accept, u_final, accept_len,
                     accept_path, next_token, ws=None, max_q_tokens=None, vocab=None, stream=None,
                     raise_on_error=True) -> int:
    """Verify drafted tokens against the target's rows ([sum n, vocab] fp32, rows any stride >= vocab apart;
    draft_probs the same, or None); writes accept_len [B], accept_path [B, width] (dense), next_token [B] (int32)."""
    batch = accept_len.shape[0]
    rows = parent.shape[0] if max_q_tokens is None else max_q_tokens
    vocab = target_probs.shape[-1] if vocab is None else vocab
    if min(t.shape[-1] for t in (target_probs, draft_probs) if t is not None) < vocab:
        raise ValueError("rows of probabilities shorter than the vocabulary")
    here = _here()
    st = lib().attn_tree_verify(int(batch), int(rows), int(vocab),
                                _vector("cu_seqlens_q", cu_seqlens_q, _int32, here, batch + 1),
                                _vector("parent", parent, _int32, here), _vector("tokens", tokens, _int32, here),
                                *_rows("target_probs", target_probs, here), *_rows("draft_probs", draft_probs, here),
                                _vector("u_accept", u_accept, _float32, here),
                                _vector("u_final", u_final, _float32, here, batch),
                                _vector("accept_len", accept_len, _int32, here), *_paths(accept_path, batch, here),
                                _vector("next_token", next_token, _int32, here, batch), _workspace(ws, here),
                                _stream_of(here, stream))
    return _check(st, "attn_tree_verify", raise_on_error)


def _rows(name, t, here):
    """Address of an fp32 matrix whose rows are dense, and the values between its rows; None is NULL."""
    if t is None:
        return None, 0
    if t.dtype is not _float32 or t.dim() != 2 or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name}: a float32 matrix with dense rows is needed")
    if t.get_device() != here:
        _elsewhere(name, t)
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[-1])


def _paths(path, batch, here):
    """Address and width of the accepted paths.  The kernels take the width for the rows' stride too and fill rows to
    it, so the rows are dense: columns inside longer rows are refused."""
    if path.dtype is not _int32 or path.dim() != 2 or path.shape[0] < batch or not path.is_contiguous():
        raise ValueError("accept_path: a dense torch.int32 matrix with a row for each request is needed")
    if path.get_device() != here:
        _elsewhere("accept_path", path)
    return path.data_ptr(), path.shape[1]


class PoolList:
    """The K/V pools of all layers, as attn_kv_compact takes them (made once, kept beside the pools)."""

    def __init__(self, pools):
        self.pools = list(pools)                    # the tensors stay alive as long as their addresses are held
        if not self.pools or self.pools[0].dim() != 3:
            raise ValueError("a list of pools [slots, Hkv, D] is needed")
        first = self.pools[0]
        self.num_slots, self.hkv, self.head_dim = (int(x) for x in first.shape)
        self.elem_bytes = first.element_size()
        for p in self.pools:
            if p.shape != first.shape or p.element_size() != self.elem_bytes or not p.is_contiguous():
                raise ValueError("the pools of a list are contiguous and of one shape and item size")
            if p.device != first.device:
                raise ValueError("the pools of a list are on one device")
        self.device = first.get_device()
        self.array = (_P * len(self.pools))(*[p.data_ptr() for p in self.pools])


def make_pool_list(pools) -> PoolList:
    """List the layers' K and V pools ([slots, Hkv, D], one shape) for attn_kv_compact."""
    return PoolList(pools)


def attn_kv_compact(pool_list, seq_lens, cu_seqlens_q, accept_len, accept_path, page_table, page_size,
                    seq_lens_out=None, ws=None, max_q_tokens=None, pt_pitch=None, stream=None,
                    raise_on_error=True) -> int:
    """Move the accepted nodes' rows behind the prefixes, in every pool of pool_list (make_pool_list);
    accept_path as attn_tree_verify writes it ([B, width], dense)."""
    batch = accept_len.shape[0]
    # only the offsets are held against the bound on the rows, so none is needed
    rows = 2 ** 31 - 1 if max_q_tokens is None else max_q_tokens
    here = _here()
    if pool_list.device != here:
        _elsewhere("pools", pool_list.pools[0])
    table, pt_pitch = _table(page_table, batch, pt_pitch, here)
    st = lib().attn_kv_compact(pool_list.array, len(pool_list.pools), pool_list.hkv, pool_list.head_dim,
                               pool_list.elem_bytes, pool_list.num_slots, int(batch), int(rows),
                               _vector("seq_lens", seq_lens, _int32, here, batch),
                               _vector("cu_seqlens_q", cu_seqlens_q, _int32, here, batch + 1),
                               _vector("accept_len", accept_len, _int32, here), *_paths(accept_path, batch, here),
                               table, pt_pitch, int(page_size),
                               _vector("seq_lens_out", seq_lens_out, _int32, here, batch), _workspace(ws, here),
                               _stream_of(here, stream))
    return _check(st, "attn_kv_compact", raise_on_error)


def pa_read_device_error(ws, stream=None) -> int:
    return lib().pa_read_device_error(_ptr(ws), _stream(stream))


def pa_noalloc_read_device_error(stream=None) -> int:
    """Read and clear the device error word of attn_decode_paged_noalloc's fixed array."""
    return lib().pa_noalloc_read_device_error(_stream(stream))


def pa_version() -> int:
    return lib().pa_version()
