"""Thin Python binding of libmla (include/mla.h): argument marshalling only.

Every function takes torch tensors that live on the current CUDA device, passes
their data pointers and the current stream to the C ABI, and raises MLAError on a
non-zero status. Importing this module loads libmla.so and raises if it is
missing: there is no other implementation behind these names. (The calls of ragged
batches, of long and common contexts and of the pages are marshalled by _binding.so and
raise if that is missing.)
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libmla.so not found at {LIB_PATH}; build it with "
        "`python -m mla_latent_kv_13_gb300.build` (needs nvcc)")

_lib = ctypes.CDLL(LIB_PATH)


class _NoBinding:
    """In the place of a _binding.so that is missing or was made for another PyTorch: the ragged
    calls, which are marshalled there, say so; the others do without it."""

    def __init__(self, why):
        self.why = why

    def __getattr__(self, name):
        def call(*args):
            raise ImportError(f"_binding.so cannot be loaded ({self.why}); build it with "
                              "`python -m mla_latent_kv_13_gb300.build` (needs nvcc and g++)")
        return call


try:
    from . import _binding  # the ragged calls' marshalling, linked to libmla.so
except ImportError as _why:
    _binding = _NoBinding(str(_why))

D_C, D_ROPE, D_QK, BLOCK, D_NOPE, D_V = 512, 64, 576, 64, 128, 128
WS_HEADER_BYTES = 256

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
          3: "MLA_ERR_WORKSPACE", 4: "MLA_ERR_OUT_OF_RANGE", 5: "MLA_ERR_TIMEOUT",
          6: "MLA_ERR_CUDA", 7: "MLA_ERR_NO_PAGES"}


class MLAError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_szp = ctypes.POINTER(ctypes.c_size_t)



class _Pool(ctypes.Structure):
    """mla_page_pool_t"""
    _fields_ = [("base", _vp), ("page_bytes", _sz), ("layer_stride", _sz), ("layers", _i)]


ROPE_MAX = 256
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class RopePlan(ctypes.Structure):
    """mla_rope_t: a rotation of `rot` values of a head. `magnitude` and `freq` may be changed."""
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("magnitude", _f),
                ("reserved", ctypes.c_int32), ("freq", ctypes.c_double * (ROPE_MAX // 2))]


_d = ctypes.c_double
_planp = ctypes.POINTER(RopePlan)

_SIGS = {
    "mla_status_string": ([_i], ctypes.c_char_p),
    "mla_append_kv_workspace_size": ([_i, _i, _szp], _i),
    "mla_append_kv": ([_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _f, _vp, _sz, _vp], _i),
    "mla_decode_workspace_size": ([_i, _i, _i, _i, _szp], _i),
    "mla_decode_plan": ([_i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)], _i),
    "mla_projection_launches": ([_i, _i, _i, _i, ctypes.POINTER(_i), ctypes.POINTER(_i),
                                 ctypes.POINTER(_i), ctypes.POINTER(_i)], _i),
    "mla_decode_schedule": ([_vp, _i, _i, _i, _vp, _i, ctypes.POINTER(_i), ctypes.POINTER(_i)],
                            _i),
    "mla_decode_attention": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _f, _i, _vp, _sz,
                              _vp, _vp, _vp], _i),
    "mla_decode_prepare": ([_vp, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "mla_decode_attention_prepared": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _f, _i, _vp,
                                       _sz, _vp, _vp, _vp], _i),
    "mla_decode_combine": ([_vp, _vp, _i, _i, _i, _vp, _vp, _vp], _i),
    "mla_decode_attention_partial": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _f, _i, _vp,
                                      _sz, _vp, _vp, _vp], _i),
    "mla_decode_combine_ranks": ([_vp, _vp, _i, _i, _i, _vp, _vp, _vp], _i),
    "mla_quantize_kv_fp8": ([_vp, ctypes.c_long, _vp, _vp, _vp], _i),
    "mla_dequantize_kv_fp8": ([_vp, _vp, ctypes.c_long, _vp, _vp], _i),
    "mla_append_kv_fp8": ([_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _vp, _i, _f, _vp, _sz, _vp], _i),
    "mla_decode_attention_fp8": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _f, _i, _vp,
                                  _sz, _vp, _vp, _vp], _i),
    "mla_decode_mq_workspace_size": ([_i, _i, _i, _i, _i, _szp], _i),
    "mla_decode_attention_mq": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _i, _f, _i, _vp,
                                 _sz, _vp, _vp, _vp], _i),
    "mla_decode_attention_noalloc": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _f, _i, _vp,
                                      _vp, _vp], _i),
    "mla_absorb_q_workspace_size": ([_i, _i, _i, _i, _szp], _i),
    "mla_absorb_q": ([_vp, _i, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _f, _vp, _sz, _vp, _vp,
                      _vp], _i),
    "mla_append_absorb_q_workspace_size": ([_i, _i, _i, _i, _szp], _i),
    "mla_append_absorb_q": ([_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp,
                             _i, _f, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_out_absorb_workspace_size": ([_i, _i, _i, _szp], _i),
    "mla_out_absorb": ([_vp, _i, _i, _vp, _vp, _i, _vp, _sz, _vp, _vp], _i),
    "mla_clear_device_status": ([_vp, _vp], _i),
    "mla_selftest_wait_timeout": ([ctypes.c_uint, _vp, _sz, _vp], _i),
    "mla_prefill_workspace_size": ([_i, _i, _i, _szp], _i),
    "mla_prefill_attention": ([_vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _vp, _vp, _f, _vp, _sz,
                               _vp, _vp, _vp], _i),
    "mla_chunk_workspace_size": ([_i, _i, _i, _i, _i, _i, _szp], _i),
    "mla_chunk_attention": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp,
                             _sz, _vp, _vp, _vp], _i),
    "mla_chunk_attention_fp8": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                 _f, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_decode_window_workspace_size": ([_i, _i, _i, _i, _i, _i, _i, _szp], _i),
    "mla_decode_attention_window": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _i, _i, _i, _f,
                                     _i, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_decode_attention_window_fp8": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _i, _i, _i, _i,
                                         _i, _f, _i, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_decode_shared_workspace_size": ([_i, _i, _i, _i, _i, _szp], _i),
    "mla_decode_attention_shared": ([_vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                     _f, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_decode_attention_shared_fp8": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _i, _i, _i,
                                         _i, _i, _f, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_norm_rope_append": ([_vp, ctypes.c_long, _i, _vp, _vp, _f, _vp, _vp, _i, _i, _vp, _i, _vp,
                              _i, _f, _vp, _vp, _sz, _vp], _i),
    "mla_norm_rope_append_fp8": ([_vp, ctypes.c_long, _i, _vp, _vp, _f, _vp, _vp, _i, _i, _vp, _i,
                                  _vp, _vp, _i, _f, _vp, _vp, _sz, _vp], _i),
    "mla_norm_rope_append_scaled": ([_vp, ctypes.c_long, _i, _vp, _vp, _f, _vp, _vp, _i, _i, _vp, _i,
                                     _vp, _i, _planp, _vp, _vp, _sz, _vp], _i),
    "mla_norm_rope_append_scaled_fp8": ([_vp, ctypes.c_long, _i, _vp, _vp, _f, _vp, _vp, _i, _i, _vp,
                                         _i, _vp, _vp, _i, _planp, _vp, _vp, _sz, _vp], _i),
    "mla_norm_rope_append_fp4": ([_vp, ctypes.c_long, _i, _vp, _vp, _f, _vp, _vp, _i, _i, _vp, _i, _vp,
                                  _vp, _vp, _vp, _i, _planp, _vp, _vp, _sz, _vp], _i),
    "mla_read_kv": ([_vp, _i, _vp, _i, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp], _i),
    "mla_read_kv_fp8": ([_vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp], _i),
    "mla_read_kv_fp4": ([_vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp], _i),
    "mla_rope_plan": ([_i, _i, _d, _i, _d, _i, _d, _d, _planp], _i),
    "mla_rope": ([_vp, ctypes.c_long, ctypes.c_long, _i, _i, _i, _i, _planp, _vp, _vp, ctypes.c_long,
                  ctypes.c_long, _vp, ctypes.c_long, ctypes.c_long, _vp], _i),
    "mla_absorb_q_latent_workspace_size": ([_i, _i, _i, _szp], _i),
    "mla_absorb_q_latent": ([_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _f, _vp, _sz, _vp, _vp, _vp], _i),
    "mla_pages_workspace_size": ([_i, _i, _szp], _i),
    "mla_pages_free": ([_vp, _i, _vp, _i, _vp, _i, _vp, _i, _vp, _sz, _vp], _i),
    "mla_pages_extend": ([_vp, _i, _vp, _i, _vp, _i, _vp, _vp, _i, _vp, _sz, _vp], _i),
    "mla_pages_fork": ([_vp, _i, _vp, _i, _vp, _i, _vp, _vp, _i, ctypes.POINTER(_Pool), _i, _vp,
                        _sz, _vp], _i),
    "mla_pages_compact": ([_vp, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, ctypes.POINTER(_Pool), _i, _vp,
                           _sz, _vp], _i),
    "mla_check_device_status": ([_vp, _vp], _i),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)


def lib():
    return _lib


def _ok(rc: int, where: str):
    if rc != 0:
        raise MLAError(rc, where)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _bits(t: torch.Tensor) -> torch.Tensor:
    """bf16 tensors pass as their 16-bit patterns; uint16/int16 views pass through."""
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"expected bf16 storage, got {t.dtype}")
    return t


def _stream(stream=None):
    if stream is None:  # the current one, without building a Stream object for each call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _size(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _ok(getattr(_lib, fn)(*args, ctypes.byref(out)), fn)
    return int(out.value)


def alloc_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """Caller-owned workspace (256-byte aligned by the caching allocator), error word cleared."""
    ws = torch.empty(max(nbytes, WS_HEADER_BYTES), dtype=torch.uint8,
                     device=device or torch.cuda.current_device())
    assert ws.data_ptr() % 256 == 0
    _ok(_lib.mla_clear_device_status(_ptr(ws), _stream(stream)), "mla_clear_device_status")
    return ws


# ------------------------------------------------------------------ sizes

def append_kv_workspace_size(B, d_model):
    return _size("mla_append_kv_workspace_size", B, d_model)


def decode_workspace_size(B, H, max_seqlen, num_splits=0):
    return _size("mla_decode_workspace_size", B, H, max_seqlen, num_splits)


def decode_plan(B, H, max_seqlen, num_splits=0):
    """(splits, launches) of mla_decode_attention for these arguments: splits = 0 for the
    balanced schedule, else the fixed token ranges per sequence."""
    s, n = _i(0), _i(0)
    rc = _lib.mla_decode_plan(B, H, max_seqlen, num_splits, ctypes.byref(s), ctypes.byref(n))
    if rc != 0:
        raise MLAError(rc, "mla_decode_plan")
    return s.value, n.value


def projection_launches(B, d_model, q_lora, H):
    """(append, absorb_q, out_absorb, append_absorb_q): the kernels one call of each
    launches for these shapes on the current device."""
    a, q, o, aq = _i(0), _i(0), _i(0), _i(0)
    rc = _lib.mla_projection_launches(B, d_model, q_lora, H, ctypes.byref(a), ctypes.byref(q),
                                      ctypes.byref(o), ctypes.byref(aq))
    if rc != 0:
        raise MLAError(rc, "mla_projection_launches")
    return a.value, q.value, o.value, aq.value


def decode_schedule(seqlens, max_blocks, clusters):
    """The balanced schedule for these lengths, computed on the host: a list of segments
    (work unit, sequence, first block, end block, part or -1 when written directly) and
    the number of fp32 parts."""
    import numpy as np
    sl = np.ascontiguousarray(seqlens, dtype=np.int32)
    cnt, parts = _i(0), _i(0)

    def call(buf, cap):
        rc = _lib.mla_decode_schedule(sl.ctypes.data_as(ctypes.c_void_p), len(sl), max_blocks,
                                      clusters, buf.ctypes.data_as(ctypes.c_void_p), cap,
                                      ctypes.byref(cnt), ctypes.byref(parts))
        if rc != 0:
            raise MLAError(rc, "mla_decode_schedule")

    call(np.zeros((1, 5), dtype=np.int32), 0)  # count only
    buf = np.zeros((max(cnt.value, 1), 5), dtype=np.int32)
    call(buf, cnt.value)
    return [tuple(int(x) for x in r) for r in buf[:cnt.value]], parts.value


def absorb_q_workspace_size(B, d_model, q_lora, H):
    return _size("mla_absorb_q_workspace_size", B, d_model, q_lora, H)


def append_absorb_q_workspace_size(B, d_model, q_lora, H):
    return _size("mla_append_absorb_q_workspace_size", B, d_model, q_lora, H)


def out_absorb_workspace_size(B, H, d_model):
    return _size("mla_out_absorb_workspace_size", B, H, d_model)


# ------------------------------------------------------------------ calls

def append_kv(h, w_dkr, pos, block_table, kv_cache, rope_theta=10000.0, workspace=None,
              stream=None):
    B, dm = h.shape
    nb = kv_cache.shape[0]
    if workspace is None:
        workspace = alloc_workspace(append_kv_workspace_size(B, dm), stream=stream)
    rc = _lib.mla_append_kv(_ptr(_bits(h)), B, dm, _ptr(_bits(w_dkr)), _ptr(pos),
                            _ptr(block_table), block_table.shape[1], _ptr(_bits(kv_cache)), nb,
                            float(rope_theta), _ptr(workspace), workspace.numel(),
                            _stream(stream))
    _ok(rc, "mla_append_kv")
    return workspace


def decode_attention(q_lat, q_rope, kv_cache, block_table, seqlens, max_seqlen, scale,
                     num_splits=0, out=None, lse=None, workspace=None, stream=None):
    """Returns (out [B,H,512] bf16, lse [B,H] fp32, workspace)."""
    B, H, _ = q_lat.shape
    dev = q_lat.device
    if out is None:
        out = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_workspace_size(B, H, max_seqlen, num_splits),
                                    stream=stream)
    rc = _lib.mla_decode_attention(_ptr(_bits(q_lat)), _ptr(_bits(q_rope)),
                                   _ptr(_bits(kv_cache)), kv_cache.shape[0], _ptr(block_table),
                                   block_table.shape[1], _ptr(seqlens), B, H, int(max_seqlen),
                                   float(scale), int(num_splits), _ptr(workspace),
                                   workspace.numel(), _ptr(out), _ptr(lse), _stream(stream))
    _ok(rc, "mla_decode_attention")
    return out, lse, workspace


def decode_prepare(seqlens, B, H, max_seqlen, num_splits, workspace, stream=None):
    """mla_decode_prepare: the balanced schedule for these lengths into the workspace (nothing
    when the plan is a fixed split), for decode_attention_prepared calls over the same
    lengths and arguments."""
    rc = _lib.mla_decode_prepare(_ptr(seqlens), int(B), int(H), int(max_seqlen), int(num_splits),
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    _ok(rc, "mla_decode_prepare")
    return workspace


def decode_attention_prepared(q_lat, q_rope, kv_cache, block_table, seqlens, max_seqlen, scale,
                              num_splits, out, lse, workspace, stream=None):
    """mla_decode_attention_prepared: decode_attention over a workspace that decode_prepare
    filled for the same lengths and arguments. Returns (out, lse, workspace)."""
    B, H, _ = q_lat.shape
    rc = _lib.mla_decode_attention_prepared(
        _ptr(_bits(q_lat)), _ptr(_bits(q_rope)), _ptr(_bits(kv_cache)), kv_cache.shape[0],
        _ptr(block_table), block_table.shape[1], _ptr(seqlens), B, H, int(max_seqlen),
        float(scale), int(num_splits), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
        _stream(stream))
    _ok(rc, "mla_decode_attention_prepared")
    return out, lse, workspace


def decode_mq_workspace_size(B, s_q, H, max_seqlen, num_splits=0):
    return _size("mla_decode_mq_workspace_size", B, s_q, H, max_seqlen, num_splits)


def decode_attention_mq(q_lat, q_rope, kv_cache, block_table, seqlens, max_seqlen, scale,
                        num_splits=0, out=None, lse=None, workspace=None, stream=None):
    """mla_decode_attention_mq: q_lat [B,s_q,H,512], q_rope [B,s_q,H,64] (draft tokens,
    causal among them). Returns (out [B,s_q,H,512] bf16, lse [B,s_q,H] fp32, workspace)."""
    B, s_q, H, _ = q_lat.shape
    dev = q_lat.device
    if out is None:
        out = torch.empty((B, s_q, H, D_C), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, s_q, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_mq_workspace_size(B, s_q, H, max_seqlen, num_splits),
                                    stream=stream)
    rc = _lib.mla_decode_attention_mq(_ptr(_bits(q_lat)), _ptr(_bits(q_rope)),
                                      _ptr(_bits(kv_cache)), kv_cache.shape[0],
                                      _ptr(block_table), block_table.shape[1], _ptr(seqlens), B,
                                      s_q, H, int(max_seqlen), float(scale), int(num_splits),
                                      _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
                                      _stream(stream))
    _ok(rc, "mla_decode_attention_mq")
    return out, lse, workspace


def decode_attention_noalloc(q_lat, q_rope, kv_cache, block_table, seqlens, max_seqlen, scale,
                             num_splits=0, out=None, lse=None, stream=None):
    """mla_decode_attention_noalloc: same results, scratch in the library's own device
    array (no workspace). Returns (out, lse)."""
    B, H, _ = q_lat.shape
    dev = q_lat.device
    if out is None:
        out = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    rc = _lib.mla_decode_attention_noalloc(_ptr(_bits(q_lat)), _ptr(_bits(q_rope)),
                                           _ptr(_bits(kv_cache)), kv_cache.shape[0],
                                           _ptr(block_table), block_table.shape[1],
                                           _ptr(seqlens), B, H, int(max_seqlen), float(scale),
                                           int(num_splits), _ptr(out), _ptr(lse),
                                           _stream(stream))
    _ok(rc, "mla_decode_attention_noalloc")
    return out, lse


def decode_combine(o_part, lse_part, out=None, lse=None, stream=None):
    B, S, H, _ = o_part.shape
    dev = o_part.device
    if out is None:
        out = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    rc = _lib.mla_decode_combine(_ptr(o_part), _ptr(lse_part), B, S, H, _ptr(out), _ptr(lse),
                                 _stream(stream))
    _ok(rc, "mla_decode_combine")
    return out, lse


def decode_attention_partial(q_lat, q_rope, kv_cache, block_table, seqlens, max_seqlen, scale,
                             num_splits=0, o_part=None, lse_part=None, workspace=None,
                             stream=None):
    """mla_decode_attention_partial: attention over this rank's token ranges only.
    Returns (o_part [B,H,512] fp32, lse_part [B,H] fp32, workspace)."""
    B, H, _ = q_lat.shape
    dev = q_lat.device
    if o_part is None:
        o_part = torch.empty((B, H, D_C), dtype=torch.float32, device=dev)
    if lse_part is None:
        lse_part = torch.empty((B, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_workspace_size(B, H, max_seqlen, num_splits),
                                    stream=stream)
    rc = _lib.mla_decode_attention_partial(_ptr(_bits(q_lat)), _ptr(_bits(q_rope)),
                                           _ptr(_bits(kv_cache)), kv_cache.shape[0],
                                           _ptr(block_table), block_table.shape[1],
                                           _ptr(seqlens), B, H, int(max_seqlen), float(scale),
                                           int(num_splits), _ptr(workspace), workspace.numel(),
                                           _ptr(o_part), _ptr(lse_part), _stream(stream))
    _ok(rc, "mla_decode_attention_partial")
    return o_part, lse_part, workspace


def decode_combine_ranks(o_parts, lse_parts, out=None, lse=None, stream=None):
    """mla_decode_combine_ranks: o_parts [G,B,H,512] fp32, lse_parts [G,B,H] fp32 ->
    (out [B,H,512] bf16, lse [B,H] fp32)."""
    G, B, H, _ = o_parts.shape
    dev = o_parts.device
    if out is None:
        out = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    rc = _lib.mla_decode_combine_ranks(_ptr(o_parts), _ptr(lse_parts), G, B, H, _ptr(out),
                                       _ptr(lse), _stream(stream))
    _ok(rc, "mla_decode_combine_ranks")
    return out, lse


def _u8(t):
    if t.dtype not in (torch.uint8, torch.int8):
        raise TypeError(f"expected 8-bit storage, got {t.dtype}")
    return t


def quantize_kv_fp8(rows_bf16, codes=None, exps=None, stream=None):
    """mla_quantize_kv_fp8: bf16 rows [..., 576] -> (codes uint8 [..., 576], exps int8 [...])."""
    shp = rows_bf16.shape
    rows = rows_bf16.numel() // D_QK
    dev = rows_bf16.device
    if codes is None:
        codes = torch.empty(shp, dtype=torch.uint8, device=dev)
    if exps is None:
        exps = torch.empty(shp[:-1], dtype=torch.int8, device=dev)
    _ok(_lib.mla_quantize_kv_fp8(_ptr(_bits(rows_bf16)), rows, _ptr(_u8(codes)), _ptr(_u8(exps)),
                                 _stream(stream)), "mla_quantize_kv_fp8")
    return codes, exps


def dequantize_kv_fp8(codes, exps, out=None, stream=None):
    """mla_dequantize_kv_fp8: (codes [..., 576], exps [...]) -> bf16 rows [..., 576]."""
    rows = codes.numel() // D_QK
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    _ok(_lib.mla_dequantize_kv_fp8(_ptr(_u8(codes)), _ptr(_u8(exps)), rows, _ptr(_bits(out)),
                                   _stream(stream)), "mla_dequantize_kv_fp8")
    return out


def append_kv_fp8(h, w_dkr, pos, block_table, kv_codes, kv_exps, rope_theta=10000.0,
                  workspace=None, stream=None):
    B, dm = h.shape
    nb = kv_codes.shape[0]
    if workspace is None:
        workspace = alloc_workspace(append_kv_workspace_size(B, dm), stream=stream)
    rc = _lib.mla_append_kv_fp8(_ptr(_bits(h)), B, dm, _ptr(_bits(w_dkr)), _ptr(pos),
                                _ptr(block_table), block_table.shape[1], _ptr(_u8(kv_codes)),
                                _ptr(_u8(kv_exps)), nb, float(rope_theta), _ptr(workspace),
                                workspace.numel(), _stream(stream))
    _ok(rc, "mla_append_kv_fp8")
    return workspace


def decode_attention_fp8(q_lat, q_rope, kv_codes, kv_exps, block_table, seqlens, max_seqlen,
                         scale, num_splits=0, out=None, lse=None, workspace=None, stream=None):
    """mla_decode_attention_fp8. Returns (out [B,H,512] bf16, lse [B,H] fp32, workspace)."""
    B, H, _ = q_lat.shape
    dev = q_lat.device
    if out is None:
        out = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_workspace_size(B, H, max_seqlen, num_splits),
                                    stream=stream)
    rc = _lib.mla_decode_attention_fp8(_ptr(_bits(q_lat)), _ptr(_bits(q_rope)),
                                       _ptr(_u8(kv_codes)), _ptr(_u8(kv_exps)), kv_codes.shape[0],
                                       _ptr(block_table), block_table.shape[1], _ptr(seqlens), B,
                                       H, int(max_seqlen), float(scale), int(num_splits),
                                       _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
                                       _stream(stream))
    _ok(rc, "mla_decode_attention_fp8")
    return out, lse, workspace


def absorb_q(h, w_dq, w_uq, w_qr, w_uk, pos, rope_theta=10000.0, q_lat=None, q_rope=None,
             workspace=None, stream=None):
    B, dm = h.shape
    ql = w_dq.shape[0]
    H = w_uk.shape[0]
    dev = h.device
    if q_lat is None:
        q_lat = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if q_rope is None:
        q_rope = torch.empty((B, H, D_ROPE), dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = alloc_workspace(absorb_q_workspace_size(B, dm, ql, H), stream=stream)
    rc = _lib.mla_absorb_q(_ptr(_bits(h)), B, dm, _ptr(_bits(w_dq)), ql, _ptr(_bits(w_uq)),
                           _ptr(_bits(w_qr)), _ptr(_bits(w_uk)), H, _ptr(pos), float(rope_theta),
                           _ptr(workspace), workspace.numel(), _ptr(q_lat), _ptr(q_rope),
                           _stream(stream))
    _ok(rc, "mla_absorb_q")
    return q_lat, q_rope, workspace


def append_absorb_q(h, w_dkr, pos, block_table, kv_cache, w_dq, w_uq, w_qr, w_uk,
                    rope_theta=10000.0, q_lat=None, q_rope=None, workspace=None, stream=None):
    """append_kv and absorb_q in one call (both read h): the new rows go into kv_cache,
    returns (q_lat, q_rope, workspace)."""
    B, dm = h.shape
    ql = w_dq.shape[0]
    H = w_uk.shape[0]
    dev = h.device
    if q_lat is None:
        q_lat = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
    if q_rope is None:
        q_rope = torch.empty((B, H, D_ROPE), dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = alloc_workspace(append_absorb_q_workspace_size(B, dm, ql, H), stream=stream)
    rc = _lib.mla_append_absorb_q(_ptr(_bits(h)), B, dm, _ptr(_bits(w_dkr)), _ptr(pos),
                                  _ptr(block_table), block_table.shape[1], _ptr(_bits(kv_cache)),
                                  kv_cache.shape[0], _ptr(_bits(w_dq)), ql, _ptr(_bits(w_uq)),
                                  _ptr(_bits(w_qr)), _ptr(_bits(w_uk)), H, float(rope_theta),
                                  _ptr(workspace), workspace.numel(), _ptr(q_lat), _ptr(q_rope),
                                  _stream(stream))
    _ok(rc, "mla_append_absorb_q")
    return q_lat, q_rope, workspace


def out_absorb(o_lat, w_uv, w_o, y=None, workspace=None, stream=None):
    B, H, _ = o_lat.shape
    dm = w_o.shape[0]
    if y is None:
        y = torch.empty((B, dm), dtype=torch.bfloat16, device=o_lat.device)
    if workspace is None:
        workspace = alloc_workspace(out_absorb_workspace_size(B, H, dm), stream=stream)
    rc = _lib.mla_out_absorb(_ptr(_bits(o_lat)), B, H, _ptr(_bits(w_uv)), _ptr(_bits(w_o)), dm,
                             _ptr(workspace), workspace.numel(), _ptr(y), _stream(stream))
    _ok(rc, "mla_out_absorb")
    return y, workspace


_arg = _binding.address  # (tensor, kind, *shape): the address, once all of it is checked
_BF16, _I32 = _binding.BF16, _binding.I32  # bf16, or its bit patterns
_pools = _binding.pools  # (caches, num_blocks): their mla_page_pool_t's


def _on(stream):
    """Buffers that a call makes belong to its stream: what fills them runs there, before the
    kernels, and their memory goes back to it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def chunk_workspace_size(B, tokens, H, max_seqlen, window=0, sinks=0):
    return _size("mla_chunk_workspace_size", B, tokens, H, int(max_seqlen), int(window), int(sinks))


def _chunk_buffers(q_lat, block_table, max_seqlen, window, sinks, out, lse, workspace, stream):
    T, H, _ = q_lat.shape
    with _on(stream):
        if out is None:
            out = torch.zeros((T, H, D_C), dtype=torch.bfloat16, device=q_lat.device)
        if lse is None:
            lse = torch.full((T, H), float("-inf"), dtype=torch.float32, device=q_lat.device)
        if workspace is None:
            workspace = alloc_workspace(
                chunk_workspace_size(block_table.shape[0], T, H, max_seqlen, window, sinks),
                stream=stream)
    return out, lse, workspace


def chunk_attention(q_lat, q_rope, kv_cache, block_table, q_starts, seqlens, max_seqlen, scale,
                    window=0, sinks=0, out=None, lse=None, workspace=None, stream=None):
    """mla_chunk_attention: q_lat [T,H,512], q_rope [T,H,64]; sequence b's new tokens are
    q_starts[b] .. q_starts[b+1]-1 (int32 [B+1]), its last ones of seqlens[b]. Rows of a padded
    batch that belong to no sequence keep what `out` and `lse` held (0 and -inf in buffers made
    here). Returns (out [T,H,512] bf16, lse [T,H] fp32, workspace)."""
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _chunk_buffers(q_lat, block_table, max_seqlen, window, sinks, out, lse,
                                             workspace, stream)
    _ok(_binding.chunk(q_lat, q_rope, kv_cache, None, block_table, q_starts, seqlens, max_seqlen, scale,
                       window, sinks, out, lse, workspace, stream), "mla_chunk_attention")
    return out, lse, workspace


def chunk_attention_fp8(q_lat, q_rope, kv_codes, kv_exps, block_table, q_starts, seqlens,
                        max_seqlen, scale, window=0, sinks=0, out=None, lse=None, workspace=None,
                        stream=None):
    """mla_chunk_attention_fp8: chunk_attention over an FP8 cache."""
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _chunk_buffers(q_lat, block_table, max_seqlen, window, sinks, out, lse,
                                             workspace, stream)
    _ok(_binding.chunk(q_lat, q_rope, kv_codes, kv_exps, block_table, q_starts, seqlens, max_seqlen,
                       scale, window, sinks, out, lse, workspace, stream), "mla_chunk_attention_fp8")
    return out, lse, workspace


def decode_window_workspace_size(B, s_q, H, max_seqlen, window, sinks=0, num_splits=0):
    return _size("mla_decode_window_workspace_size", B, s_q, H, int(max_seqlen), int(window),
                 int(sinks), int(num_splits))


def _window_buffers(q_lat, max_seqlen, window, sinks, num_splits, out, lse, workspace, stream):
    lead, H = q_lat.shape[:-2], q_lat.shape[-2]  # (B,) or (B, s_q)
    with _on(stream):
        if out is None:
            out = torch.empty((*lead, H, D_C), dtype=torch.bfloat16, device=q_lat.device)
        if lse is None:
            lse = torch.empty((*lead, H), dtype=torch.float32, device=q_lat.device)
        if workspace is None:
            workspace = alloc_workspace(
                decode_window_workspace_size(lead[0], lead[1] if len(lead) > 1 else 1, H, max_seqlen,
                                             window, sinks, num_splits), stream=stream)
    return out, lse, workspace


def decode_attention_window(q_lat, q_rope, kv_cache, block_table, seqlens, max_seqlen, window,
                            sinks, scale, num_splits=0, out=None, lse=None, workspace=None,
                            stream=None):
    """mla_decode_attention_window: q_lat [B,H,512] or [B,s_q,H,512] (draft tokens, causal among
    them); a token at position p sees the rows j <= p with j > p - window or j < sinks. Returns
    (out bf16, lse fp32, workspace) in the layout of q_lat."""
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _window_buffers(q_lat, max_seqlen, window, sinks, num_splits, out, lse,
                                              workspace, stream)
    _ok(_binding.window(q_lat, q_rope, kv_cache, None, block_table, seqlens, max_seqlen, window, sinks,
                        scale, num_splits, out, lse, workspace, stream),
        "mla_decode_attention_window")
    return out, lse, workspace


def decode_attention_window_fp8(q_lat, q_rope, kv_codes, kv_exps, block_table, seqlens,
                                max_seqlen, window, sinks, scale, num_splits=0, out=None,
                                lse=None, workspace=None, stream=None):
    """mla_decode_attention_window_fp8: decode_attention_window over an FP8 cache."""
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _window_buffers(q_lat, max_seqlen, window, sinks, num_splits, out, lse,
                                              workspace, stream)
    _ok(_binding.window(q_lat, q_rope, kv_codes, kv_exps, block_table, seqlens, max_seqlen, window,
                        sinks, scale, num_splits, out, lse, workspace, stream),
        "mla_decode_attention_window_fp8")
    return out, lse, workspace


def decode_shared_workspace_size(B, s_q, H, max_seqlen, groups):
    return _size("mla_decode_shared_workspace_size", B, s_q, H, int(max_seqlen), int(groups))


def _shared_buffers(q_lat, max_seqlen, prefix_lens, out, lse, workspace, stream):
    lead, H = q_lat.shape[:-2], q_lat.shape[-2]  # (B,) or (B, s_q)
    with _on(stream):
        if out is None:
            out = torch.empty((*lead, H, D_C), dtype=torch.bfloat16, device=q_lat.device)
        if lse is None:
            lse = torch.empty((*lead, H), dtype=torch.float32, device=q_lat.device)
        if workspace is None:
            workspace = alloc_workspace(
                decode_shared_workspace_size(lead[0], lead[1] if len(lead) > 1 else 1, H, max_seqlen,
                                             prefix_lens.shape[0]), stream=stream)
    return out, lse, workspace


def decode_attention_shared(q_lat, q_rope, kv_cache, block_table, seqlens, group_starts,
                            prefix_lens, max_seqlen, scale, out=None, lse=None, workspace=None,
                            stream=None):
    """mla_decode_attention_shared: decode attention (q_lat [B,H,512] or [B,s_q,H,512], draft tokens
    causal among them) where the sequences group_starts[g] .. group_starts[g+1]-1 hold the same pages
    for their first prefix_lens[g] // 64 ones (int32 [G+1] and [G]). Returns (out bf16, lse fp32,
    workspace) in the layout of q_lat."""
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _shared_buffers(q_lat, max_seqlen, prefix_lens, out, lse, workspace,
                                              stream)
    _ok(_binding.shared(q_lat, q_rope, kv_cache, None, block_table, seqlens, group_starts, prefix_lens,
                        max_seqlen, scale, out, lse, workspace, stream),
        "mla_decode_attention_shared")
    return out, lse, workspace


def decode_attention_shared_fp8(q_lat, q_rope, kv_codes, kv_exps, block_table, seqlens,
                                group_starts, prefix_lens, max_seqlen, scale, out=None, lse=None,
                                workspace=None, stream=None):
    """mla_decode_attention_shared_fp8: decode_attention_shared over an FP8 cache."""
    if out is None or lse is None or workspace is None:
        out, lse, workspace = _shared_buffers(q_lat, max_seqlen, prefix_lens, out, lse, workspace,
                                              stream)
    _ok(_binding.shared(q_lat, q_rope, kv_codes, kv_exps, block_table, seqlens, group_starts,
                        prefix_lens, max_seqlen, scale, out, lse, workspace, stream),
        "mla_decode_attention_shared_fp8")
    return out, lse, workspace


def _norm_buffers(x, c_q, workspace, stream):
    if not x.is_cuda:
        raise ValueError("x: a CUDA tensor of bf16 rows [tokens, q_lora + 576]")
    with _on(stream):
        if c_q is None:
            T, width = x.shape
            c_q = torch.zeros((T, max(width - D_QK, 0)), dtype=torch.bfloat16, device=x.device)
        if workspace is None:
            workspace = alloc_workspace(WS_HEADER_BYTES, stream=stream)
    return c_q, workspace


def norm_rope_append(x, w_q, w_kv, q_starts, seqlens, block_table, kv_cache, rope_theta=10000.0,
                     eps=1e-6, c_q=None, workspace=None, stream=None):
    """mla_norm_rope_append: x [T, q_lora + 576] (rows may be strided), the new tokens of a ragged
    batch as in chunk_attention. Returns (c_q [T, q_lora] bf16, workspace); the normed, rotated
    keys go into kv_cache."""
    if c_q is None or workspace is None:
        c_q, workspace = _norm_buffers(x, c_q, workspace, stream)
    _ok(_binding.norm(x, w_q, w_kv, q_starts, seqlens, block_table, kv_cache, None, rope_theta, eps,
                      c_q, workspace, stream), "mla_norm_rope_append")
    return c_q, workspace


def norm_rope_append_fp8(x, w_q, w_kv, q_starts, seqlens, block_table, kv_codes, kv_exps,
                         rope_theta=10000.0, eps=1e-6, c_q=None, workspace=None, stream=None):
    """mla_norm_rope_append_fp8: norm_rope_append into an FP8 cache."""
    if c_q is None or workspace is None:
        c_q, workspace = _norm_buffers(x, c_q, workspace, stream)
    _ok(_binding.norm(x, w_q, w_kv, q_starts, seqlens, block_table, kv_codes, kv_exps, rope_theta, eps,
                      c_q, workspace, stream), "mla_norm_rope_append_fp8")
    return c_q, workspace


def norm_rope_append_scaled(x, w_q, w_kv, q_starts, seqlens, block_table, kv_cache, plan, eps=1e-6,
                            c_q=None, workspace=None, stream=None):
    """mla_norm_rope_append_scaled: norm_rope_append with a plan's rotation (rope_plan, rot = 64)."""
    if c_q is None or workspace is None:
        c_q, workspace = _norm_buffers(x, c_q, workspace, stream)
    _ok(_binding.norm_plan(x, w_q, w_kv, q_starts, seqlens, block_table, kv_cache, None, None, None,
                           plan, eps, c_q, workspace, stream), "mla_norm_rope_append_scaled")
    return c_q, workspace


def norm_rope_append_scaled_fp8(x, w_q, w_kv, q_starts, seqlens, block_table, kv_codes, kv_exps, plan,
                                eps=1e-6, c_q=None, workspace=None, stream=None):
    """mla_norm_rope_append_scaled_fp8: norm_rope_append_scaled into an FP8 cache."""
    if c_q is None or workspace is None:
        c_q, workspace = _norm_buffers(x, c_q, workspace, stream)
    _ok(_binding.norm_plan(x, w_q, w_kv, q_starts, seqlens, block_table, kv_codes, kv_exps, None, None,
                           plan, eps, c_q, workspace, stream), "mla_norm_rope_append_scaled_fp8")
    return c_q, workspace


def norm_rope_append_fp4(x, w_q, w_kv, q_starts, seqlens, block_table, kv_codes, kv_scales, kv_exps,
                         kv_keys, plan, eps=1e-6, c_q=None, workspace=None, stream=None):
    """mla_norm_rope_append_fp4: norm_rope_append_scaled into a 4-bit cache: kv_codes [num_blocks, 64,
    256], kv_scales [num_blocks, 64, 32] uint8, kv_exps [num_blocks, 64] int8, kv_keys [num_blocks, 64,
    64] bf16."""
    if c_q is None or workspace is None:
        c_q, workspace = _norm_buffers(x, c_q, workspace, stream)
    _ok(_binding.norm_plan(x, w_q, w_kv, q_starts, seqlens, block_table, kv_codes, kv_exps, kv_scales,
                           kv_keys, plan, eps, c_q, workspace, stream), "mla_norm_rope_append_fp4")
    return c_q, workspace


def rope_plan(rot=D_ROPE, theta=10000.0, scaling="none", factor=1.0, original=4096, fast=32.0,
              slow=1.0, layout="interleaved", magnitude=None):
    """mla_rope_plan: the rotation of `rot` values of a head as a RopePlan, its frequencies scaled as
    "none", "linear", "ntk", "yarn" or "bands" says (include/mla.h); magnitude: another one than the
    scaling's."""
    plan = RopePlan()
    if scaling not in ROPE_SCALINGS or layout not in ROPE_LAYOUTS:
        raise ValueError(f"scaling is one of {list(ROPE_SCALINGS)}, layout one of {list(ROPE_LAYOUTS)}")
    _ok(_lib.mla_rope_plan(int(rot), ROPE_LAYOUTS[layout], float(theta), ROPE_SCALINGS[scaling],
                           float(factor), int(original), float(fast), float(slow),
                           ctypes.byref(plan)), "mla_rope_plan")
    if magnitude is not None:
        plan.magnitude = magnitude
    return plan


def rope(x, pos, plan, offset=0, out=None, rest=None, split=False, stream=None):
    """mla_rope: x [T,H,width] (strided, last dimension contiguous) with the values offset ..
    offset + plan.rot - 1 of each head rotated at pos [T] int32, into out [T,H,rot], which may be that
    place itself: out=x[..., offset:offset + plan.rot]. rest [T,H,width - rot] gets the others (made
    here with split). Returns out, or (out, rest) where there is a rest."""
    if not isinstance(plan, RopePlan):
        raise TypeError("expected what rope_plan() gave")
    if out is None or (rest is None and split):
        with _on(stream):
            if out is None:
                out = torch.empty((*x.shape[:2], plan.rot), dtype=torch.bfloat16, device=x.device)
            if rest is None and split:
                rest = torch.empty((*x.shape[:2], x.shape[2] - plan.rot), dtype=torch.bfloat16,
                                   device=x.device)
    _ok(_binding.rope(x, pos, plan, offset, out, rest, stream), "mla_rope")
    return out if rest is None else (out, rest)


def _read_buffers(block_table, rows, out, workspace, stream):
    with _on(stream):
        if out is None:
            if rows is None:
                raise ValueError("rows or out is wanted")
            out = torch.zeros((rows, D_QK), dtype=torch.bfloat16, device=block_table.device)
        if workspace is None:
            workspace = alloc_workspace(WS_HEADER_BYTES, stream=stream)
    return out, workspace


def read_kv(kv_cache, block_table, first, row_starts, rows=None, out=None, workspace=None,
            stream=None):
    """mla_read_kv: sequence b's cached rows from first[b] on (int32 [B]; None: 0) to the rows
    row_starts[b] .. row_starts[b+1]-1 of out [rows, 576] bf16. Returns (out, workspace)."""
    if out is None or workspace is None:
        out, workspace = _read_buffers(block_table, rows, out, workspace, stream)
    _ok(_binding.read(kv_cache, None, None, None, block_table, first, row_starts, out, workspace,
                      stream), "mla_read_kv")
    return out, workspace


def read_kv_fp8(kv_codes, kv_exps, block_table, first, row_starts, rows=None, out=None,
                workspace=None, stream=None):
    """mla_read_kv_fp8: read_kv from an FP8 cache (exact)."""
    if out is None or workspace is None:
        out, workspace = _read_buffers(block_table, rows, out, workspace, stream)
    _ok(_binding.read(kv_codes, kv_exps, None, None, block_table, first, row_starts, out, workspace,
                      stream), "mla_read_kv_fp8")
    return out, workspace


def read_kv_fp4(kv_codes, kv_scales, kv_exps, kv_keys, block_table, first, row_starts, rows=None,
                out=None, workspace=None, stream=None):
    """mla_read_kv_fp4: read_kv from a 4-bit cache (exact)."""
    if out is None or workspace is None:
        out, workspace = _read_buffers(block_table, rows, out, workspace, stream)
    _ok(_binding.read(kv_codes, kv_exps, kv_scales, kv_keys, block_table, first, row_starts, out,
                      workspace, stream), "mla_read_kv_fp4")
    return out, workspace


def absorb_q_latent_workspace_size(B, q_lora, H):
    return _size("mla_absorb_q_latent_workspace_size", B, q_lora, H)


def absorb_q_latent(c_q, w_uq, w_qr, w_uk, pos, rope_theta=10000.0, q_lat=None, q_rope=None,
                    workspace=None, stream=None):
    """mla_absorb_q_latent: absorb_q from the (normed) query latent c_q [B, q_lora] on."""
    B, ql = c_q.shape
    H = w_uk.shape[0]
    dev = c_q.device
    if q_lat is None or q_rope is None or workspace is None:
        with _on(stream):
            if q_lat is None:
                q_lat = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
            if q_rope is None:
                q_rope = torch.empty((B, H, D_ROPE), dtype=torch.bfloat16, device=dev)
            if workspace is None:
                workspace = alloc_workspace(absorb_q_latent_workspace_size(B, ql, H), stream=stream)
    rc = _lib.mla_absorb_q_latent(_arg(c_q, _BF16, B, ql), B, ql, _ptr(_bits(w_uq)), _ptr(_bits(w_qr)),
                                  _ptr(_bits(w_uk)), H, _arg(pos, _I32, B), float(rope_theta),
                                  _ptr(workspace), workspace.numel(), _arg(q_lat, _BF16, B, H, D_C),
                                  _arg(q_rope, _BF16, B, H, D_ROPE), _stream(stream))
    _ok(rc, "mla_absorb_q_latent")
    return q_lat, q_rope, workspace


def pages_workspace_size(num_blocks, num_seqs):
    return _size("mla_pages_workspace_size", num_blocks, num_seqs)


def _pages_buffer(refs, block_table, stream):
    with _on(stream):
        return alloc_workspace(pages_workspace_size(refs.shape[0], block_table.shape[0]),
                               stream=stream)


def pages_free(refs, block_table, seqlens, rows, workspace=None, stream=None):
    """mla_pages_free: the rows release their pages. refs [num_blocks], block_table [num_seqs,
    max_blocks], seqlens [num_seqs] int32 are updated. Returns the workspace."""
    if workspace is None:
        workspace = _pages_buffer(refs, block_table, stream)
    _ok(_binding.pages_free(refs, block_table, seqlens, rows, workspace, stream), "mla_pages_free")
    return workspace


def pages_extend(refs, block_table, seqlens, rows, new_lens, workspace=None, stream=None):
    """mla_pages_extend: the rows grow to new_lens, taking the lowest free pages."""
    if workspace is None:
        workspace = _pages_buffer(refs, block_table, stream)
    _ok(_binding.pages_extend(refs, block_table, seqlens, rows, new_lens, workspace, stream),
        "mla_pages_extend")
    return workspace


def pages_fork(refs, block_table, seqlens, parents, children, pools, workspace=None, stream=None):
    """mla_pages_fork: empty rows become copies of their parents. pools: the caches
    [layers, num_blocks, ...] whose partial pages are copied (kv_cache[None] for one layer; codes
    and exps of an FP8 cache); layers may be strided, a layer is contiguous."""
    if workspace is None:
        workspace = _pages_buffer(refs, block_table, stream)
    _ok(_binding.pages_fork(refs, block_table, seqlens, parents, children,
                            _pools(pools, refs.shape[0]), workspace, stream), "mla_pages_fork")
    return workspace


def pages_compact(refs, block_table, seqlens, pools, refs_out=None, table_out=None, live=None,
                  workspace=None, stream=None):
    """mla_pages_compact: live pages move to the pool's front, in every pool; refs and block_table
    are rewritten in place unless refs_out / table_out are given. Returns (refs_out, table_out,
    live [1] int32: the number of live pages, workspace)."""
    if workspace is None:
        workspace = _pages_buffer(refs, block_table, stream)
    refs_out = refs if refs_out is None else refs_out
    table_out = block_table if table_out is None else table_out
    if live is None:
        with _on(stream):
            live = torch.empty(1, dtype=torch.int32, device=refs.device)
    _ok(_binding.pages_compact(refs, block_table, seqlens, _pools(pools, refs.shape[0]), refs_out,
                               table_out, live, workspace, stream), "mla_pages_compact")
    return refs_out, table_out, live, workspace


def check_device_status(workspace, stream=None) -> int:
    """Synchronise and return (and clear) the workspace's device error word."""
    return int(_lib.mla_check_device_status(_ptr(workspace), _stream(stream)))


def prefill_workspace_size(H, prefix, chunk):
    return _size("mla_prefill_workspace_size", H, prefix, chunk)


def prefill_attention(q_nope, q_rope, kv_cache, block_table_row, prefix, w_uk, w_uv, scale,
                      out=None, lse=None, workspace=None, stream=None):
    """mla_prefill_attention: q_nope [C,H,128], q_rope [C,H,64] of one sequence's chunk at
    positions prefix.. (already appended). Returns (out [C,H,128] bf16, lse [C,H] fp32,
    workspace)."""
    C, H, _ = q_nope.shape
    dev = q_nope.device
    if out is None:
        out = torch.empty((C, H, D_V), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((C, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(prefill_workspace_size(H, prefix, C), stream=stream)
    rc = _lib.mla_prefill_attention(_ptr(_bits(q_nope)), _ptr(_bits(q_rope)),
                                    _ptr(_bits(kv_cache)), kv_cache.shape[0],
                                    _ptr(block_table_row), block_table_row.numel(), int(prefix),
                                    C, H, _ptr(_bits(w_uk)), _ptr(_bits(w_uv)), float(scale),
                                    _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
                                    _stream(stream))
    _ok(rc, "mla_prefill_attention")
    return out, lse, workspace


def selftest_wait_timeout(limit_us, workspace, stream=None):
    """Run the failure-detection self-test; returns (status, detail) from the workspace
    header after it (expected: MLA_ERR_TIMEOUT and at least limit_us microseconds)."""
    _ok(_lib.mla_selftest_wait_timeout(int(limit_us), _ptr(workspace), workspace.numel(),
                                       _stream(stream)), "mla_selftest_wait_timeout")
    torch.cuda.synchronize(workspace.device)
    hdr = workspace[:8].view(torch.int32).cpu().tolist()
    return hdr[0] & 0xFFFFFFFF, hdr[1] & 0xFFFFFFFF


def clear_device_status(workspace, stream=None):
    _ok(_lib.mla_clear_device_status(_ptr(workspace), _stream(stream)), "mla_clear_device_status")


class DecodeStep:
    """The absorbed MLA decode step for one layer: append the new token's latent,
    build the absorbed query, attend over the paged cache, project the latent
    output back. Holds caller-owned workspaces; every step runs in libmla kernels."""

    def __init__(self, weights: dict, B: int, H: int, max_seqlen: int, num_splits: int = 0,
                 rope_theta: float = 10000.0, scale: float | None = None):
        self.w = weights
        self.B, self.H = B, H
        self.dm = weights["w_dkr"].shape[1]
        self.ql = weights["w_dq"].shape[0]
        self.max_seqlen = max_seqlen
        self.num_splits = num_splits
        self.theta = rope_theta
        self.scale = (1.0 / (D_NOPE + D_ROPE) ** 0.5) if scale is None else scale
        dev = weights["w_dkr"].device
        self.ws_q = alloc_workspace(append_absorb_q_workspace_size(B, self.dm, self.ql, H))
        self.ws_att = alloc_workspace(decode_workspace_size(B, H, max_seqlen, num_splits))
        self.ws_out = alloc_workspace(out_absorb_workspace_size(B, H, self.dm))
        self.q_lat = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
        self.q_rope = torch.empty((B, H, D_ROPE), dtype=torch.bfloat16, device=dev)
        self.o_lat = torch.empty((B, H, D_C), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((B, H), dtype=torch.float32, device=dev)
        self.y = torch.empty((B, self.dm), dtype=torch.bfloat16, device=dev)

    def __call__(self, h, pos, seqlens_after, block_table, kv_cache, stream=None, out=None):
        """One step; the result y [B, d_model] bf16 goes to `out` if given, else to the
        step's own buffer (returned either way). One stream: the new cache rows and the
        absorbed query (one call: both read h), the attention schedule (it reads only the
        lengths, so it runs beside the last query projection), the attention, the output
        projections."""
        w = self.w
        y = self.y if out is None else out
        main = torch.cuda.current_stream() if stream is None else stream
        append_absorb_q(h, w["w_dkr"], pos, block_table, kv_cache, w["w_dq"], w["w_uq"],
                        w["w_qr"], w["w_uk"], self.theta, self.q_lat, self.q_rope, self.ws_q,
                        main)
        decode_prepare(seqlens_after, self.B, self.H, self.max_seqlen, self.num_splits,
                       self.ws_att, main)
        decode_attention_prepared(self.q_lat, self.q_rope, kv_cache, block_table, seqlens_after,
                                  self.max_seqlen, self.scale, self.num_splits, self.o_lat,
                                  self.lse, self.ws_att, main)
        out_absorb(self.o_lat, w["w_uv"], w["w_o"], y, self.ws_out, main)
        return y

    def check(self, stream=None) -> int:
        codes = [check_device_status(ws, stream) for ws in (self.ws_q, self.ws_att, self.ws_out)]
        return next((c for c in codes if c), 0)
