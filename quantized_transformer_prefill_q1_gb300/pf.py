"""ctypes binding of libpf (include/pf.h): the same entry-point names, argument
marshalling only. Every step of the path runs in libpf's CUDA kernels; torch is used
for device memory and streams. If libpf.so is missing, importing the library raises —
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpf.so")

PF_OK = 0
STATUS = {
    0: "PF_OK", 1: "PF_ERR_INVALID_ARG", 2: "PF_ERR_SHAPE", 3: "PF_ERR_EMPTY_CHUNK",
    4: "PF_ERR_NONSEQUENTIAL_START", 5: "PF_ERR_TOKEN_OUT_OF_VOCAB", 6: "PF_ERR_KV_CAPACITY",
    7: "PF_ERR_LOGITS", 8: "PF_ERR_UNSUPPORTED", 9: "PF_ERR_CUDA", 10: "PF_ERR_DEVICE_TIMEOUT",
    11: "PF_ERR_WORKSPACE", 12: "PF_ERR_NONFINITE",
}
W_Q1, W_INT4 = 0, 1
KV_F32, KV_BF16, KV_F16, KV_E4M3, KV_INT8 = 0, 1, 2, 3, 4
EPI_STORE_F32, EPI_RESID_ADD, EPI_SWIGLU = 0, 1, 2
KERNEL_CLASSES = ("rmsnorm", "gemm_qkv", "qk_rope_kv", "attention", "gemm_o", "gemm_gate_up",
                  "gemm_down", "embed", "lm_head", "other")
_WFMT = {"q1": W_Q1, "int4": W_INT4}
_KVDT = {"f32": KV_F32, "bf16": KV_BF16, "f16": KV_F16, "e4m3": KV_E4M3, "int8": KV_INT8}


class PfError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class pf_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("eps", ctypes.c_float), ("final_eps", ctypes.c_float),
                ("qk_norm", ctypes.c_int32), ("wfmt", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("max_seq", ctypes.c_int32),
                ("max_chunk", ctypes.c_int32), ("ring_capacity", ctypes.c_int32),
                ("sink_count", ctypes.c_int32), ("kv_block_pool", ctypes.c_int32)]

KV_BLOCK = 128  # PF_KV_BLOCK: positions per paged KV block
KV8_BLOCK = 32  # PF_KV8_BLOCK: slots that share one scale in an 8-bit cache
MAX_TOP = 32    # PF_MAX_TOP: most alternatives per row of pf_op_logprobs
MAX_SEQS = 1024  # PF_MAX_SEQS: most sequences of a batch
MAX_TREE = 256   # PF_MAX_TREE: most rows of one sequence with a tree
MAX_RANK = 128   # PF_MAX_RANK: largest adapter rank


class pf_layer_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("attn_norm", "qkv", "q_norm", "k_norm", "o_proj", "ffn_norm", "gate_up", "down")]


class pf_model(ctypes.Structure):
    _fields_ = [("cfg", pf_config), ("layers", ctypes.POINTER(pf_layer_weights)),
                ("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p),
                ("lm_head", ctypes.c_void_p)]


class pf_batch(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("row_begin_dev", ctypes.c_void_p), ("start_dev", ctypes.c_void_p),
                ("parent_dev", ctypes.c_void_p), ("block_table_dev", ctypes.c_void_p)]


_VP, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "pf_last_error": ([], ctypes.c_char_p),
    "pf_status_name": ([ctypes.c_int], ctypes.c_char_p),
    "pf_abi_version": ([], _I32),
    "pf_packed_bytes": ([_I32, _I64, _I64], _SZ),
    "pf_pack_weights_host": ([_I32, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _SZ], _I32),
    "pf_kv_bytes": ([ctypes.POINTER(pf_config)], _SZ),
    "pf_workspace_bytes": ([ctypes.POINTER(pf_config)], _SZ),
    "pf_config_check": ([ctypes.POINTER(pf_config)], _I32),
    "pf_validate_chunk": ([ctypes.POINTER(pf_config), _I32, _VP, _I32, _I32, _I32, _I32], _I32),
    "pf_session_create": ([ctypes.POINTER(pf_model), _VP, _VP, _VP, _SZ, _VP,
                           ctypes.POINTER(_VP)], _I32),
    "pf_session_destroy": ([_VP], _I32),
    "pf_session_position": ([_VP], _I32),
    "pf_session_set_position": ([_VP, _I32], _I32),
    "pf_session_set_graphs": ([_VP, _I32], _I32),
    "pf_session_set_block_table": ([_VP, _VP, _I32], _I32),
    "pf_session_sync": ([_VP, _VP], _I32),
    "pf_prefill_chunk": ([_VP, _VP, _I32, _I32, _VP, _VP], _I32),
    "pf_prefill_chunk_dev": ([_VP, _VP, _I32, _I32, _VP, _VP], _I32),
    "pf_decode_step": ([_VP, _VP, _VP, _VP], _I32),
    "pf_decode_step_greedy": ([_VP, _VP, _VP, _VP, _VP], _I32),
    "pf_prefill_verify": ([_VP, _VP, _I32, _I32, _VP, _VP, _VP], _I32),
    "pf_session_set_profile": ([_VP, _I32], _I32),
    "pf_session_profile_read": ([_VP, _VP, ctypes.POINTER(ctypes.c_double),
                                 ctypes.POINTER(ctypes.c_int64)], _I32),
    "pf_session_kernel_launches": ([_VP], ctypes.c_int64),
    "pf_timeline_set": ([_VP, ctypes.c_int64], _I32),
    "pf_timeline_kernel_name": ([_I32], ctypes.c_char_p),
    "pf_prefill_hidden": ([_VP, _VP, _I32, _I32, _VP, _VP], _I32),
    "pf_layer_forward": ([_VP, _I32, _VP, _I32, _I32, _VP], _I32),
    "pf_prefill_tokens_host": ([_VP, _VP, _I32, _I32, _VP, _VP], _I32),
    "pf_op_rmsnorm": ([_VP, _VP, _F, _I32, _I32, _VP, _VP], _I32),
    "pf_op_dequant": ([_I32, _VP, _I64, _I64, _VP, _VP], _I32),
    "pf_op_gemm": ([_I32, _I32, _VP, _VP, _I32, _I32, _I32, _VP, _I32, _VP, _SZ, _VP, _VP], _I32),
    "pf_gemm_scratch_bytes": ([_I32, _I32, _I32], _SZ),
    "pf_op_gemm_static_scratch": ([_I32, _I32, _VP, _VP, _I32, _I32, _I32, _VP, _VP, _VP], _I32),
    "pf_streamk_plan_host": ([_I32, _I32, _I32, _I32, _I32, _I32, _VP, _VP, _I32, _VP, _I32, _VP], _I32),
    "pf_op_qk_norm_rope_kv": ([ctypes.POINTER(pf_config), _VP, _VP, _VP, _VP, _I32, _I32, _I32,
                               _VP, _VP, _VP, _VP], _I32),
    "pf_op_attention": ([ctypes.POINTER(pf_config), _VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP], _I32),
    "pf_attention_scratch_bytes": ([ctypes.POINTER(pf_config), _I32, _I32], _SZ),
    "pf_op_attention_split": ([ctypes.POINTER(pf_config), _VP, _VP, _VP, _I32, _I32, _I32, _I32, _VP, _SZ,
                               _VP, _VP], _I32),
    "pf_op_embed": ([_VP, _VP, _I32, _I32, _I32, _VP, _VP, _VP], _I32),
    "pf_op_lm_head": ([_I32, _VP, _VP, _F, _VP, _I32, _I32, _VP, _VP], _I32),
    "pf_op_argmax": ([_VP, _I32, _I32, _I64, _VP, _VP], _I32),
    "pf_rope_table_host": ([_F, _I32, _I32, _VP], _I32),
    "pf_op_logprobs": ([_VP, _I32, _I32, _I64, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP], _I32),
    "pf_prefill_score": ([_VP, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _I32, _VP, _VP, _VP], _I32),
    "pf_kv8_scales_offset": ([ctypes.POINTER(pf_config)], _SZ),
    "pf_op_kv8_store": ([ctypes.POINTER(pf_config), _VP, _VP, _I64, _I64, _I32, _I32, _I32, _VP, _VP, _VP, _VP,
                         _VP], _I32),
    "pf_op_kv8_load": ([ctypes.POINTER(pf_config), _VP, _I32, _I32, _I32, _VP, _VP, _VP, _VP], _I32),
    "pf_attention_kv8_scratch_bytes": ([ctypes.POINTER(pf_config), _I32], _SZ),
    "pf_op_attention_kv8": ([ctypes.POINTER(pf_config), _VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP, _VP, _SZ, _VP,
                             _VP], _I32),
    "pf_op_batch_append": ([ctypes.POINTER(pf_config), ctypes.POINTER(pf_batch), _VP, _VP, _VP, _VP, _I32, _VP, _VP,
                            _VP, _VP, _VP], _I32),
    "pf_attention_tree_scratch_bytes": ([ctypes.POINTER(pf_config), _I32, _I32], _SZ),
    "pf_op_attention_tree": ([ctypes.POINTER(pf_config), ctypes.POINTER(pf_batch), _VP, _VP, _VP, _I32, _VP, _VP, _SZ,
                              _VP, _VP], _I32),
    "pf_op_tree_accept": ([ctypes.POINTER(pf_config), ctypes.POINTER(pf_batch), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                           _VP, _VP], _I32),
    "pf_op_adapters": ([ctypes.POINTER(pf_batch), _VP, _I64, _VP, _I64, _VP, _I64, _I32, _I32, _I32, _I32, _VP, _VP, _VP,
                        _VP, _VP, _VP], _I32),
    "pf_status_read": ([_VP, _VP], _I32),
    "pf_selftest_bounded_wait": ([_VP, _I64, _I32, _VP], _I32),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Loads libpf.so (built by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpf.so not built ({LIB_PATH}); run __graft_entry__.build()")
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _lib = l
    return _lib


def header_symbols() -> List[str]:
    return list(_SIGS)


def check(status: int) -> None:
    if status != PF_OK:
        raise PfError(status, lib().pf_last_error().decode())


def _ptr(t) -> Optional[int]:
    """Device / host address of a torch tensor or numpy array (None passes NULL)."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        assert t.flags["C_CONTIGUOUS"]
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream=None) -> Optional[int]:
    if stream is not None:
        return stream
    import torch
    # the current stream's handle without a Stream object around it (0.1 us instead of 2.8)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


# ------------------------------------------------------------------ host-side calls
def make_config(shape, max_chunk: int, n_layers: Optional[int] = None, max_seq: Optional[int] = None,
                vocab: Optional[int] = None, ring_capacity: int = 0, sink_count: int = 0,
                kv_block_pool: int = 0) -> pf_config:
    return pf_config(hidden=shape.hidden, intermediate=shape.intermediate,
                     n_q_heads=shape.n_q_heads, n_kv_heads=shape.n_kv_heads,
                     head_dim=shape.head_dim,
                     n_layers=shape.n_layers if n_layers is None else n_layers,
                     vocab=shape.vocab if vocab is None else vocab,
                     rope_theta=shape.rope_theta, eps=shape.eps, final_eps=shape.final_eps,
                     qk_norm=int(shape.qk_norm), wfmt=_WFMT[shape.wfmt],
                     kv_dtype=_KVDT[shape.kv_dtype],
                     max_seq=shape.max_seq if max_seq is None else max_seq, max_chunk=max_chunk,
                     ring_capacity=ring_capacity, sink_count=sink_count, kv_block_pool=kv_block_pool)


def pf_packed_bytes(wfmt: int, n: int, k: int) -> int:
    return lib().pf_packed_bytes(wfmt, n, k)


def pf_pack_weights_host(w: Dict, interleave_gate_up: bool = False) -> np.ndarray:
    """Packs one canonical quantised tensor (see ``synth``) into libpf's device layout."""
    wfmt = _WFMT[w["fmt"]]
    n, k = w["n"], w["k"]
    nbytes = pf_packed_bytes(wfmt, n, k)
    out = np.empty(nbytes, np.uint8)
    codes = np.ascontiguousarray(w["bits"] if wfmt == W_Q1 else w["codes"])
    scales = np.ascontiguousarray(w["scales"]).view(np.uint16)
    zeros = None if wfmt == W_Q1 else np.ascontiguousarray(w["zeros"]).view(np.uint16)
    check(lib().pf_pack_weights_host(wfmt, _ptr(codes), _ptr(scales), _ptr(zeros), n, k,
                                     int(interleave_gate_up), _ptr(out), nbytes))
    return out


def pf_validate_chunk(cfg: pf_config, kv_position: int, tokens: Optional[np.ndarray], m: int,
                      start: int, want_logits: bool, has_head: bool) -> int:
    t = None if tokens is None else np.ascontiguousarray(tokens, dtype=np.int32)
    return lib().pf_validate_chunk(ctypes.byref(cfg), kv_position, _ptr(t), m, start,
                                   int(want_logits), int(has_head))


def pf_rope_table_host(theta: float, head_dim: int, max_seq: int) -> np.ndarray:
    out = np.empty((max_seq, head_dim // 2, 2), np.float32)
    check(lib().pf_rope_table_host(theta, head_dim, max_seq, _ptr(out)))
    return out


# ------------------------------------------------------------------ single steps (GPU)
def pf_op_rmsnorm(x, w, eps, y, stream=None):
    m, h = x.shape
    check(lib().pf_op_rmsnorm(_ptr(x), _ptr(w), eps, m, h, _ptr(y), _stream(stream)))


def pf_op_dequant(wfmt, packed, n, k, out, stream=None):
    check(lib().pf_op_dequant(wfmt, _ptr(packed), n, k, _ptr(out), _stream(stream)))


def pf_gemm_scratch_bytes(m, n, max_ctas=0):
    return lib().pf_gemm_scratch_bytes(m, n, max_ctas)


def gemm_scratch(m, n, max_ctas=0, device="cuda"):
    """Zeroed scratch (uint8 tensor) for pf_op_gemm on an M x N output."""
    import torch
    return torch.zeros(pf_gemm_scratch_bytes(m, n, max_ctas), dtype=torch.uint8, device=device)


def pf_op_gemm(wfmt, epilogue, a, packed, m, n, k, out, scratch, max_ctas=0, status=None,
               stream=None):
    check(lib().pf_op_gemm(wfmt, epilogue, _ptr(a), _ptr(packed), m, n, k, _ptr(out), max_ctas,
                           _ptr(scratch), scratch.numel() * scratch.element_size(), _ptr(status),
                           _stream(stream)))


def pf_op_gemm_static_scratch(wfmt, epilogue, a, packed, m, n, k, out, status=None, stream=None):
    """pf_op_gemm with the library's fixed scratch: for callers that may not allocate."""
    check(lib().pf_op_gemm_static_scratch(wfmt, epilogue, _ptr(a), _ptr(packed), m, n, k, _ptr(out),
                                          _ptr(status), _stream(stream)))


def pf_streamk_plan_host(n_mt, n_nt, kbt, ctas, late_units=0, late_kb=0, max_segs=8, w_query=None):
    """The GEMMs' stream-K partition on the host: (begins [ctas + 1], segments [ctas, max_segs, 4]
    as (tile, kb0, nkb, slot; -1 slot for a whole tile; tile -1 past the last), owners of
    w_query or None)."""
    begins = np.zeros(ctas + 1, np.int64)
    segs = np.zeros((ctas, max_segs, 4), np.int32)
    wq = None if w_query is None else np.ascontiguousarray(w_query, np.int64)
    owners = None if wq is None else np.zeros(len(wq), np.int32)
    check(lib().pf_streamk_plan_host(n_mt, n_nt, kbt, ctas, late_units, late_kb, _ptr(begins), _ptr(segs),
                                     max_segs, _ptr(wq), 0 if wq is None else len(wq), _ptr(owners)))
    return begins, segs, owners


def pf_op_qk_norm_rope_kv(cfg, qkv, qn, kn, rope, layer, start, m, q, kc, vc, stream=None):
    check(lib().pf_op_qk_norm_rope_kv(ctypes.byref(cfg), _ptr(qkv), _ptr(qn), _ptr(kn), _ptr(rope),
                                      layer, start, m, _ptr(q), _ptr(kc), _ptr(vc), _stream(stream)))


def pf_op_attention(cfg, q, kc, vc, layer, start, m, out, stream=None):
    check(lib().pf_op_attention(ctypes.byref(cfg), _ptr(q), _ptr(kc), _ptr(vc), layer, start, m,
                                _ptr(out), _stream(stream)))


def pf_attention_scratch_bytes(cfg, m, n_split):
    return lib().pf_attention_scratch_bytes(ctypes.byref(cfg), m, n_split)


def pf_op_attention_split(cfg, q, kc, vc, layer, start, m, n_split, scratch, out, stream=None):
    check(lib().pf_op_attention_split(ctypes.byref(cfg), _ptr(q), _ptr(kc), _ptr(vc), layer, start, m,
                                      n_split, _ptr(scratch), scratch.numel() * scratch.element_size(),
                                      _ptr(out), _stream(stream)))


def pf_op_argmax(x, rows, n, ld, out, stream=None):
    check(lib().pf_op_argmax(_ptr(x), rows, n, ld, _ptr(out), _stream(stream)))


# Operators over the 8-bit cache and the logits: the tensors' device, type and layout are checked
# here (PF_ERR_INVALID_ARG), everything else by the library. These are small calls: the checks read
# a tensor's fields only (about 0.3 us a tensor).
_torch = None


def _here():
    """Index of the current CUDA device (no tensor's without a GPU), as a function fixed on first use."""
    global _torch, _here
    import torch
    _torch = torch
    if torch.cuda.is_available():
        torch.cuda.current_device()  # initialises CUDA
        _here = torch._C._cuda_getDevice
    else:
        _here = lambda: -2  # noqa: E731
    return _here()


def _dense(t, dev: int, dtype: str, what: str, numel: int, optional: bool = False) -> Optional[int]:
    """Address of a contiguous tensor of CUDA device `dev` holding at least numel elements."""
    if t is None:
        if optional:
            return None
        raise PfError(1, f"{what} is None")
    if t.get_device() == dev and t.dtype is getattr(_torch, dtype) and t.numel() >= numel and t.is_contiguous():
        return t.data_ptr()
    if t.get_device() != dev:
        raise PfError(1, f"{what} is on {t.device}, not on the current CUDA device")
    raise PfError(1, f"{what}: need at least {numel} contiguous {dtype} elements, got {tuple(t.shape)} {t.dtype}")


def _rows(t, dev: int, what: str, rows: int, n: int, ld: int) -> Optional[int]:
    """Address of f32 rows of n values, ld apart: a view [>= rows, >= n] of such strides, or contiguous elements."""
    if t is not None and t.dim() == 2 and t.shape[0] >= rows and t.shape[1] >= n:
        st = t.stride()
        if ((st[0] == ld or rows == 1) and (st[1] == 1 or n == 1) and t.get_device() == dev and t.dtype is _torch.float32):
            return t.data_ptr()
    return _dense(t, dev, "float32", what, (rows - 1) * ld + n)


def _on(dev: int, stream) -> Optional[int]:
    """The stream, or the current one of CUDA device `dev`."""
    return stream if stream is not None else _torch._C._cuda_getCurrentRawStream(dev)


def _is_kv8(cfg) -> bool:
    return cfg.kv_dtype in (KV_E4M3, KV_INT8)


def _table(cfg, dev: int, blocks) -> Optional[int]:
    return None if blocks is None else _dense(blocks, dev, "int32", "block table", -(-cfg.max_seq // KV_BLOCK))


def kv8_cache(cfg, device="cuda"):
    """One zeroed 8-bit cache buffer (K or V): codes, then scales."""
    import torch
    check(lib().pf_config_check(ctypes.byref(cfg)))
    return torch.zeros(lib().pf_kv_bytes(ctypes.byref(cfg)), dtype=torch.uint8, device=device)


def kv8_views(cfg, cache):
    """(codes [n_layers, nkv, slots, hd] float8_e4m3fn / int8, scales [n_layers, nkv, blocks] f32)
    of one 8-bit cache buffer, as views of it."""
    import torch
    at = lib().pf_kv8_scales_offset(ctypes.byref(cfg))
    if at == 0:
        raise PfError(8, f"kv dtype {cfg.kv_dtype} is not an 8-bit type")
    slots = cfg.kv_block_pool * KV_BLOCK if cfg.kv_block_pool > 0 else cfg.max_seq
    n = cfg.n_layers * cfg.n_kv_heads * slots * cfg.head_dim
    code = torch.float8_e4m3fn if cfg.kv_dtype == KV_E4M3 else torch.int8
    nblk = -(-slots // KV8_BLOCK)
    scales = cache[at:at + 4 * cfg.n_layers * cfg.n_kv_heads * nblk].view(torch.float32)
    return (cache[:n].view(code).view(cfg.n_layers, cfg.n_kv_heads, slots, cfg.head_dim),
            scales.view(cfg.n_layers, cfg.n_kv_heads, nblk))


def pf_op_kv8_store(cfg, k, v, layer, start, m, k_cache, v_cache, blocks=None, status=None, stream=None):
    """k, v: f16 [m, nkv, hd], any token and head strides (multiples of 8, the same for both; those of a
    dimension of 1 do not count)."""
    dev, l, ref = _here(), lib(), ctypes.byref(cfg)
    nkv = cfg.n_kv_heads
    st, sv = k.stride(), v.stride()
    if (k.get_device() != dev or v.get_device() != dev or k.dtype is not _torch.float16 or v.dtype is not _torch.float16
            or k.shape != (m, nkv, cfg.head_dim) or v.shape != k.shape or st[2] != 1 or sv[2] != 1
            or (m > 1 and sv[0] != st[0]) or (nkv > 1 and sv[1] != st[1])):
        raise PfError(1, f"K / V rows: need f16 {(m, nkv, cfg.head_dim)} of equal strides with contiguous elements "
                         f"on the current CUDA device, got {[(tuple(t.shape), t.dtype, t.stride(), str(t.device)) for t in (k, v)]}")
    n = l.pf_kv_bytes(ref)
    check(l.pf_op_kv8_store(ref, k.data_ptr(), v.data_ptr(), st[0] if m > 1 else 0, st[1] if nkv > 1 else 0, layer, start, m, _table(cfg, dev, blocks),
                            _dense(k_cache, dev, "uint8", "K cache", n), _dense(v_cache, dev, "uint8", "V cache", n),
                            _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def pf_op_kv8_load(cfg, cache, layer, start, m, out, blocks=None, status=None, stream=None):
    """out: f32 [m, nkv, hd], the values that one cache (K or V) holds at positions start .. start + m - 1."""
    dev, l, ref = _here(), lib(), ctypes.byref(cfg)
    check(l.pf_op_kv8_load(ref, _dense(cache, dev, "uint8", "cache", l.pf_kv_bytes(ref)), layer, start, m, _table(cfg, dev, blocks),
                           _dense(out, dev, "float32", "out", m * cfg.n_kv_heads * cfg.head_dim),
                           _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def pf_attention_kv8_scratch_bytes(cfg, m):
    return lib().pf_attention_kv8_scratch_bytes(ctypes.byref(cfg), m)


def attention_kv8_scratch(cfg, m, device="cuda"):
    """Scratch (uint8 tensor, its counters zeroed) for pf_op_attention_kv8 on up to m tokens."""
    import torch
    check(lib().pf_config_check(ctypes.byref(cfg)))
    return torch.zeros(pf_attention_kv8_scratch_bytes(cfg, m), dtype=torch.uint8, device=device)


def pf_op_attention_kv8(cfg, q, k_cache, v_cache, layer, start, m, out, scratch, blocks=None, status=None,
                        stream=None):
    """Causal attention of q f16 [m, nq, hd] over the 8-bit caches, into out f16 [m, nq * hd]."""
    dev, l, ref = _here(), lib(), ctypes.byref(cfg)
    n, nc = m * cfg.n_q_heads * cfg.head_dim, l.pf_kv_bytes(ref)
    check(l.pf_op_attention_kv8(ref, _dense(q, dev, "float16", "q", n), _dense(k_cache, dev, "uint8", "K cache", nc),
                                _dense(v_cache, dev, "uint8", "V cache", nc), layer, start, m, _table(cfg, dev, blocks),
                                _dense(out, dev, "float16", "out", n), _dense(scratch, dev, "uint8", "scratch", 0),
                                scratch.numel(), _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def pf_op_logprobs(logits, rows, n, ld, tokens, logprobs, entropy=None, top=0, top_ids=None, top_logprobs=None,
                   status=None, stream=None):
    """Log probability of tokens[r], entropy and the top alternatives of each row of logits [rows, ld], or of a
    view [rows, n] whose rows are ld apart (each output may be None)."""
    dev = _here()
    check(lib().pf_op_logprobs(_rows(logits, dev, "logits", rows, n, ld), rows, n, ld,
                               _dense(tokens, dev, "int32", "tokens", rows, True),
                               _dense(logprobs, dev, "float32", "logprobs", rows, True),
                               _dense(entropy, dev, "float32", "entropy", rows, True), top,
                               _dense(top_ids, dev, "int32", "top_ids", rows * top, True),
                               _dense(top_logprobs, dev, "float32", "top_logprobs", rows * top, True),
                               _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


class Batch:
    """The rows of a step over many sequences (pf_batch): row_begin int32 [n_seq + 1] on the device, start int32 [n_seq],
    parent int32 [n_rows] (None: chains), blocks int32 [n_seq, pages] (paged caches). n_rows: rows that the row arrays
    hold; max_rows: most rows of one sequence. The tensors' contents may change from step to step; the tensors
    themselves are kept alive here and checked here, once."""

    def __init__(self, row_begin, n_rows: int, max_rows: int, start=None, parent=None, blocks=None):
        self.device = dev = _here()
        if row_begin is None or row_begin.dim() != 1 or row_begin.shape[0] < 2:
            raise PfError(1, "row_begin: need int32 [n_seq + 1]")
        n_seq = row_begin.shape[0] - 1
        if blocks is not None and (blocks.dim() != 2 or blocks.shape[0] != n_seq):
            raise PfError(1, f"blocks: need int32 [{n_seq}, pages], got {tuple(blocks.shape)}")
        self.pages = 0 if blocks is None else blocks.shape[1]
        self.keep = (row_begin, start, parent, blocks)
        self.n_seq, self.n_rows = n_seq, n_rows
        self.c = pf_batch(n_seq=n_seq, n_rows=n_rows, max_rows=max_rows,
                          row_begin_dev=_dense(row_begin, dev, "int32", "row_begin", n_seq + 1),
                          start_dev=_dense(start, dev, "int32", "start", n_seq, True),
                          parent_dev=_dense(parent, dev, "int32", "parent", n_rows, True),
                          block_table_dev=_dense(blocks, dev, "int32", "blocks", n_seq, True))
        self.ref = ctypes.byref(self.c)


def _batch(batch, dev: int, cfg=None):
    """The batch's struct for a call on CUDA device `dev` (with a configuration: over its caches)."""
    if batch.device != dev:
        raise PfError(1, f"the batch is on cuda:{batch.device}, not on the current CUDA device")
    if cfg is not None and cfg.kv_block_pool > 0 and batch.pages and batch.pages != -(-cfg.max_seq // KV_BLOCK):
        raise PfError(1, f"blocks: need {-(-cfg.max_seq // KV_BLOCK)} entries a sequence, got {batch.pages}")
    return batch.ref


def _caches16(cfg, dev: int, k, v):
    """Addresses of a 16-bit K and V cache buffer of the configuration's type."""
    pool = cfg.kv_block_pool
    n = cfg.n_layers * cfg.n_kv_heads * (pool * KV_BLOCK if pool > 0 else cfg.max_seq) * cfg.head_dim
    dt = _KV_TORCH.get(cfg.kv_dtype, "float16")
    return _dense(k, dev, dt, "K cache", n), _dense(v, dev, dt, "V cache", n)


def pf_op_batch_append(cfg, batch, qkv, qn, kn, rope, layer, q, k_cache, v_cache, status=None, stream=None):
    """QK-norm, RoPE and KV store of every sequence's rows: qkv f32 [n_rows, (nq + 2 nkv) hd], q of the cache's type
    [n_rows, nq, hd], rope f32 [max_seq, hd / 2, 2] on the device (pf_rope_table_host)."""
    dev, n, hd, nq = _here(), batch.n_rows, cfg.head_dim, cfg.n_q_heads
    k, v = _caches16(cfg, dev, k_cache, v_cache)
    check(lib().pf_op_batch_append(ctypes.byref(cfg), _batch(batch, dev, cfg),
                                   _dense(qkv, dev, "float32", "qkv", n * (nq + 2 * cfg.n_kv_heads) * hd),
                                   _dense(qn, dev, "float32", "q_norm", hd, True), _dense(kn, dev, "float32", "k_norm", hd, True),
                                   _dense(rope, dev, "float32", "rope", cfg.max_seq * hd), layer,
                                   _dense(q, dev, _KV_TORCH.get(cfg.kv_dtype, "float16"), "q", n * nq * hd), k, v,
                                   _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def pf_attention_tree_scratch_bytes(cfg, n_seq, max_rows):
    return lib().pf_attention_tree_scratch_bytes(ctypes.byref(cfg), n_seq, max_rows)


def attention_tree_scratch(cfg, n_seq, max_rows, device="cuda"):
    """Zeroed scratch (uint8 tensor) for pf_op_attention_tree on up to n_seq sequences of up to max_rows rows."""
    import torch
    check(lib().pf_config_check(ctypes.byref(cfg)))
    n = pf_attention_tree_scratch_bytes(cfg, n_seq, max_rows)
    if n == 0:
        raise PfError(2, f"n_seq {n_seq}: 1..{MAX_SEQS}; max_rows {max_rows}: 1..{MAX_TREE}")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def pf_op_attention_tree(cfg, batch, q, k_cache, v_cache, layer, out, scratch, status=None, stream=None):
    """Attention of every sequence's rows over the cache: q of the cache's type [n_rows, nq, hd], out f16 [n_rows, nq * hd]."""
    dev = _here()
    n = batch.n_rows * cfg.n_q_heads * cfg.head_dim
    k, v = _caches16(cfg, dev, k_cache, v_cache)
    check(lib().pf_op_attention_tree(ctypes.byref(cfg), _batch(batch, dev, cfg),
                                     _dense(q, dev, _KV_TORCH.get(cfg.kv_dtype, "float16"), "q", n), k, v, layer,
                                     _dense(out, dev, "float16", "out", n), _dense(scratch, dev, "uint8", "scratch", 0),
                                     scratch.numel(), _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def pf_op_tree_accept(cfg, batch, tokens, ids, root_ids, path, n_accepted, next_ids, k_cache=None, v_cache=None, status=None,
                      stream=None):
    """Greedy acceptance of each sequence's tree (int32: tokens, ids, path [n_rows]; root_ids, n_accepted, next_ids
    [n_seq]); the accepted nodes' K and V move up in every layer of the caches (None: nothing is moved)."""
    dev, n, b = _here(), batch.n_rows, batch.n_seq
    if (k_cache is None) != (v_cache is None):
        raise PfError(1, "both caches or none")
    k, v = (None, None) if k_cache is None else _caches16(cfg, dev, k_cache, v_cache)
    check(lib().pf_op_tree_accept(ctypes.byref(cfg), _batch(batch, dev, cfg), _dense(tokens, dev, "int32", "tokens", n),
                                  _dense(ids, dev, "int32", "ids", n), _dense(root_ids, dev, "int32", "root_ids", b),
                                  _dense(path, dev, "int32", "path", n), _dense(n_accepted, dev, "int32", "n_accepted", b),
                                  _dense(next_ids, dev, "int32", "next_ids", b), k, v,
                                  _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def _strided(t, dev: int, dtype: str, what: str, rows: int, width: int):
    """(address, elements between rows) of rows [>= rows, width] with contiguous elements."""
    if t is None or t.dim() != 2:
        raise PfError(1, f"{what}: need {dtype} [{rows}, {width}], got {None if t is None else tuple(t.shape)}")
    (n, w), (apart, step) = t.shape, t.stride()
    if n < rows or w != width:
        raise PfError(1, f"{what}: need {dtype} [{rows}, {width}], got {tuple(t.shape)}")
    if t.get_device() != dev or t.dtype is not getattr(_torch, dtype) or (step != 1 and w != 1):
        raise PfError(1, f"{what}: need {dtype} rows with contiguous elements on the current CUDA device, got {t.dtype} "
                         f"of strides {t.stride()} on {t.device}")
    return t.data_ptr(), apart if rows > 1 else -(-w // 8) * 8


def pf_op_adapters(batch, x, base, out, adapter, a, b, scale, status=None, stream=None):
    """out[m] = base[m] + scale[i] (x[m] A_i^T) B_i^T with i = adapter[sequence of m], -1: none. x f16 [n_rows, K], base and
    out f32 [n_rows, N] (views of wider rows; out may be base), a f16 [adapters, rank, K], b f16 [adapters, N, rank],
    scale f32 [adapters], adapter int32 [n_seq]."""
    dev, rows = _here(), batch.n_rows
    if a is None or b is None or a.dim() != 3 or b.dim() != 3:
        raise PfError(1, "A: need f16 [adapters, rank, K], B: f16 [adapters, N, rank]")
    (count, rank, k), (others, n, r) = a.shape, b.shape
    if others != count or r != rank:
        raise PfError(1, f"A {(count, rank, k)} and B {(others, n, r)}: need [adapters, rank, K] and [adapters, N, rank]")
    xp, ldx = _strided(x, dev, "float16", "x", rows, k)
    bp, ldb = _strided(base, dev, "float32", "base", rows, n)
    op, ldo = (bp, ldb) if out is base else _strided(out, dev, "float32", "out", rows, n)
    check(lib().pf_op_adapters(_batch(batch, dev), xp, ldx, bp, ldb, op, ldo, k, n, rank, count,
                               _dense(adapter, dev, "int32", "adapter", batch.n_seq), _dense(a, dev, "float16", "A", count * rank * k),
                               _dense(b, dev, "float16", "B", count * n * rank), _dense(scale, dev, "float32", "scale", count),
                               _dense(status, dev, "int32", "status", 1, True), _on(dev, stream)))


def pf_op_embed(e, tokens, m, h, vocab, x, status=None, stream=None):
    check(lib().pf_op_embed(_ptr(e), _ptr(tokens), m, h, vocab, _ptr(x), _ptr(status),
                            _stream(stream)))


def pf_op_lm_head(wfmt, x_row, norm_w, eps, packed, vocab, h, logits, stream=None):
    check(lib().pf_op_lm_head(wfmt, _ptr(x_row), _ptr(norm_w), eps, _ptr(packed), vocab, h,
                              _ptr(logits), _stream(stream)))


def pf_status_read(status, stream=None):
    check(lib().pf_status_read(_ptr(status), _stream(stream)))


def pf_selftest_bounded_wait(status, limit_ns: int, arrive: bool, stream=None):
    check(lib().pf_selftest_bounded_wait(_ptr(status), limit_ns, int(arrive), _stream(stream)))


# ------------------------------------------------------------------ model + session
def pf_timeline_set(buffer, capacity: int) -> None:
    """Point every libpf kernel's per-CTA timeline at `buffer` (device int64/uint64 tensor
    of 4 + 4 * capacity words), or stop recording with None."""
    check(lib().pf_timeline_set(_ptr(buffer), int(capacity) if buffer is not None else 0))


def pf_timeline_kernel_name(kernel_id: int) -> Optional[str]:
    n = lib().pf_timeline_kernel_name(int(kernel_id))
    return n.decode() if n is not None else None


def timeline_records(buffer) -> np.ndarray:
    """The records of a timeline buffer as a structured array (start_ns, end_ns, kernel,
    sm, cta), sorted by start; records past the capacity were dropped by the device."""
    b = buffer.cpu().numpy().view(np.uint64)
    n = int(min(b[0], b[1]))
    r = b[4:4 + 4 * n].reshape(n, 4)
    out = np.zeros(n, dtype=[("start_ns", np.int64), ("end_ns", np.int64), ("kernel", np.int32),
                             ("sm", np.int32), ("cta", np.int64)])
    out["start_ns"] = r[:, 0].astype(np.int64)
    out["end_ns"] = r[:, 1].astype(np.int64)
    out["kernel"] = (r[:, 2] >> np.uint64(48)).astype(np.int32)
    out["sm"] = ((r[:, 2] >> np.uint64(32)) & np.uint64(0xffff)).astype(np.int32)
    out["cta"] = (r[:, 2] & np.uint64(0xffffffff)).astype(np.int64)
    return np.sort(out, order="start_ns", kind="stable")


class DeviceModel:
    """Uploads a stack's weights (packed once, on the host) into device memory owned by
    torch tensors and fills a ``pf_model`` pointing at them."""

    def __init__(self, shape, layers: Sequence[Dict], extra: Optional[Dict] = None,
                 max_chunk: int = 512, device: str = "cuda", max_seq: Optional[int] = None,
                 ring_capacity: int = 0, sink_count: int = 0, kv_block_pool: int = 0):
        import torch
        self.shape = shape
        self.keep: List = []
        extra = extra or {}

        def dev(a: np.ndarray):
            t = torch.from_numpy(np.ascontiguousarray(a)).to(device)
            self.keep.append(t)
            return t

        def packed(w, inter=False):
            return dev(pf_pack_weights_host(w, inter))

        n = len(layers)
        self.cfg = make_config(shape, max_chunk, n_layers=n, max_seq=max_seq,
                               vocab=shape.vocab if "lm_head" in extra else 0,
                               ring_capacity=ring_capacity, sink_count=sink_count,
                               kv_block_pool=kv_block_pool)
        self.layer_arr = (pf_layer_weights * n)()
        for i, w in enumerate(layers):
            lw = self.layer_arr[i]
            lw.attn_norm = _ptr(dev(w["attn_norm"]))
            lw.ffn_norm = _ptr(dev(w["ffn_norm"]))
            lw.q_norm = _ptr(dev(w["q_norm"])) if w["q_norm"] is not None else None
            lw.k_norm = _ptr(dev(w["k_norm"])) if w["k_norm"] is not None else None
            lw.qkv = _ptr(packed(w["qkv"]))
            lw.o_proj = _ptr(packed(w["o"]))
            lw.gate_up = _ptr(packed(w["gate_up"], True))
            lw.down = _ptr(packed(w["down"]))
        self.model = pf_model(cfg=self.cfg, layers=self.layer_arr)
        if "embed" in extra:
            self.model.embed = _ptr(dev(extra["embed"]))
        if "lm_head" in extra:
            self.model.final_norm = _ptr(dev(extra["final_norm"]))
            self.model.lm_head = _ptr(packed(extra["lm_head"]))


_KV_TORCH = {KV_F32: "float32", KV_BF16: "bfloat16", KV_F16: "float16", KV_E4M3: "uint8", KV_INT8: "uint8"}


class Session:
    """A pf_session with its KV cache and workspace allocated by torch (caller-owned)."""

    def __init__(self, dm: DeviceModel, stream=None, kv_fill_bits: Optional[int] = None,
                 graphs: bool = True, kv=None, block_table: Optional[Sequence[int]] = None):
        """`kv`: an existing (k, v) pair to share (paged caches: one pool, disjoint block
        tables); `block_table`: a paged session's table (default: position block b in
        physical block b, when the pool has enough blocks)."""
        import torch
        self.dm = dm
        c = dm.cfg
        dt = getattr(torch, _KV_TORCH[c.kv_dtype])
        slots = c.ring_capacity if c.ring_capacity > 0 else (
            c.kv_block_pool * KV_BLOCK if c.kv_block_pool > 0 else c.max_seq)
        shape = (c.n_layers, c.n_kv_heads, slots, c.head_dim)
        if _is_kv8(c):  # codes and scales in one buffer (kv8_views)
            shape = (lib().pf_kv_bytes(ctypes.byref(c)),)
        if kv is not None:
            self.k, self.v = kv
        else:
            self.k = torch.empty(shape, dtype=dt, device="cuda")
            self.v = torch.empty(shape, dtype=dt, device="cuda")
        if kv_fill_bits is not None:  # sentinel bit pattern in every slot
            ib = torch.int32 if c.kv_dtype == KV_F32 else torch.int16
            self.k.view(ib).fill_(kv_fill_bits)
            self.v.view(ib).fill_(kv_fill_bits)
        check(lib().pf_config_check(ctypes.byref(c)))
        wsb = lib().pf_workspace_bytes(ctypes.byref(c))
        if wsb == 0:
            raise PfError(2, lib().pf_last_error().decode())
        self.ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
        h = ctypes.c_void_p()
        check(lib().pf_session_create(ctypes.byref(dm.model), _ptr(self.k), _ptr(self.v),
                                      _ptr(self.ws), wsb, _stream(stream), ctypes.byref(h)))
        self.h = h
        check(lib().pf_session_set_graphs(self.h, int(graphs)))
        if c.kv_block_pool > 0:
            n = -(-c.max_seq // KV_BLOCK)
            if block_table is None and c.kv_block_pool >= n:
                block_table = range(n)
            if block_table is not None:
                self.set_block_table(block_table)

    def set_block_table(self, table: Sequence[int]) -> None:
        t = np.ascontiguousarray(np.asarray(table, dtype=np.int32))
        check(lib().pf_session_set_block_table(self.h, _ptr(t), len(t)))

    @property
    def position(self) -> int:
        return lib().pf_session_position(self.h)

    def set_position(self, p: int) -> None:
        check(lib().pf_session_set_position(self.h, p))

    def set_graphs(self, on: bool) -> None:
        check(lib().pf_session_set_graphs(self.h, int(on)))

    def prefill_chunk(self, tokens: np.ndarray, start: int, logits=None, stream=None) -> None:
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        check(lib().pf_prefill_chunk(self.h, _ptr(t), len(t), start, _ptr(logits), _stream(stream)))

    def prefill_chunk_dev(self, tokens_dev, start: int, logits=None, stream=None) -> None:
        check(lib().pf_prefill_chunk_dev(self.h, _ptr(tokens_dev), tokens_dev.shape[0], start,
                                         _ptr(logits), _stream(stream)))

    def decode_step(self, token_dev, logits, stream=None) -> None:
        """One decode step: the token at token_dev (device int32) at the current position."""
        check(lib().pf_decode_step(self.h, _ptr(token_dev), _ptr(logits), _stream(stream)))

    def decode_step_greedy(self, token_in_dev, token_out_dev, logits, stream=None) -> None:
        """A decode step whose logits' argmax (device int32) is written to token_out_dev."""
        check(lib().pf_decode_step_greedy(self.h, _ptr(token_in_dev), _ptr(token_out_dev), _ptr(logits),
                                          _stream(stream)))

    def prefill_verify(self, tokens_dev, start: int, logits_all, ids, stream=None) -> None:
        """Prefill of tokens_dev, then logits [M, vocab] and their argmax [M] at every position."""
        check(lib().pf_prefill_verify(self.h, _ptr(tokens_dev), tokens_dev.shape[0], start, _ptr(logits_all),
                                      _ptr(ids), _stream(stream)))

    def prefill_score(self, tokens_dev, targets_dev, start: int, logits_all, logprobs, entropy=None, top: int = 0,
                      top_ids=None, top_logprobs=None, stream=None) -> None:
        """Prefill of tokens_dev, logits [M, vocab] at every position, then pf_op_logprobs of targets_dev [M]."""
        m, dev = tokens_dev.shape[0], _here()
        check(lib().pf_prefill_score(self.h, _dense(tokens_dev, dev, "int32", "tokens", m),
                                     _dense(targets_dev, dev, "int32", "targets", m), m, start,
                                     _dense(logits_all, dev, "float32", "logits", m * self.dm.cfg.vocab),
                                     _dense(logprobs, dev, "float32", "logprobs", m),
                                     _dense(entropy, dev, "float32", "entropy", m, True), top,
                                     _dense(top_ids, dev, "int32", "top_ids", m * top, True),
                                     _dense(top_logprobs, dev, "float32", "top_logprobs", m * top, True),
                                     _on(dev, stream)))

    def set_profile(self, on: bool) -> None:
        check(lib().pf_session_set_profile(self.h, int(on)))

    def profile_read(self, stream=None) -> Dict[str, tuple]:
        """{kernel class: (summed ms, launches)} since the previous read."""
        ms = (ctypes.c_double * len(KERNEL_CLASSES))()
        n = (ctypes.c_int64 * len(KERNEL_CLASSES))()
        check(lib().pf_session_profile_read(self.h, _stream(stream), ms, n))
        return {name: (ms[i], n[i]) for i, name in enumerate(KERNEL_CLASSES)}

    @property
    def kernel_launches(self) -> int:
        return lib().pf_session_kernel_launches(self.h)

    def prefill_hidden(self, x, start: int, logits=None, stream=None) -> None:
        check(lib().pf_prefill_hidden(self.h, _ptr(x), x.shape[0], start, _ptr(logits),
                                      _stream(stream)))

    def layer_forward(self, layer: int, x, start: int, stream=None) -> None:
        check(lib().pf_layer_forward(self.h, layer, _ptr(x), x.shape[0], start, _stream(stream)))

    def prefill_tokens_host(self, tokens: np.ndarray, start: int, logits_host: Optional[np.ndarray],
                            stream=None) -> None:
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        check(lib().pf_prefill_tokens_host(self.h, _ptr(t), len(t), start, _ptr(logits_host),
                                           _stream(stream)))

    def sync(self, stream=None) -> None:
        check(lib().pf_session_sync(self.h, _stream(stream)))

    def close(self) -> None:
        if getattr(self, "h", None):
            lib().pf_session_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
