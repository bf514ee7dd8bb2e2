"""Thin ctypes binding of libmamba_state.so (argument marshalling only).

Every function here has the name of the C entry point it calls, takes torch CUDA tensors (or
None for nullable arguments), passes their device pointers and sizes, and raises
:class:`MambaError` on a non-zero status.  All arithmetic happens in the CUDA kernels; there is
no CPU path.  Loading fails loudly when the library has not been built.

Layouts are the ones the C header documents (include/mamba_state.h); tensors must be
contiguous except the pools, whose slot stride is taken from ``stride(0)``.  Each tensor's
dtype is checked against the layer descriptor before its pointer is passed (ValueError), since
the C ABI sees only addresses.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import workloads as wl

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmamba_state.so")

MAMBA_OK, MAMBA_EINVAL, MAMBA_EUNSUPPORTED, MAMBA_ECUDA, MAMBA_EALIGN, MAMBA_ENOSPACE = 0, -1, -2, -3, -4, -5
MAMBA_F32, MAMBA_BF16 = 0, 1
MAMBA_ERR_SLOT_RANGE, MAMBA_ERR_ACCEPT_RANGE, MAMBA_ERR_SEQLENS, MAMBA_ERR_TIMEOUT = 0x1, 0x2, 0x4, 0x8


class MambaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class LayerDesc(ctypes.Structure):
    """Mirror of ``mamba_layer_desc``."""

    _fields_ = [(n, ctypes.c_int32) for n in ("nheads", "head_dim", "d_state", "n_groups", "conv_kernel",
                                              "num_spec", "state_dtype", "conv_dtype", "act_dtype",
                                              "dt_dtype")]


class Mamba1Desc(ctypes.Structure):
    """Mirror of ``mamba1_layer_desc``."""

    _fields_ = [(n, ctypes.c_int32) for n in ("d_inner", "d_state", "conv_kernel", "num_spec", "state_dtype",
                                              "conv_dtype", "act_dtype", "dt_dtype")]


def mamba1_desc(d_inner: int, d_state: int, conv_kernel: int = 4, num_spec: int = 0, state: str = wl.BF16,
                act: str = wl.BF16, dt: str = wl.F32) -> Mamba1Desc:
    code = wl.DTYPE_CODE
    return Mamba1Desc(d_inner, d_state, conv_kernel, num_spec, code[state], code[act], code[act], code[dt])


def layer_desc(shape: "wl.LayerShape", state: str = wl.BF16, act: str = wl.BF16, dt: str = wl.F32,
               conv: str | None = None) -> LayerDesc:
    code = wl.DTYPE_CODE
    return LayerDesc(shape.nheads, shape.head_dim, shape.d_state, shape.n_groups, shape.conv_kernel,
                     shape.num_spec, code[state], code[conv or act], code[act], code[dt])


_lock = threading.Lock()
_lib = None
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_f32 = ctypes.c_float
_dp = ctypes.POINTER(LayerDesc)
_d1 = ctypes.POINTER(Mamba1Desc)

# (name, restype, argtypes) of every exported entry point
SIGNATURES = {
    "mamba_conv_dim": (_i32, [_dp]),
    "mamba_ssm_state_bytes": (_i64, [_dp]),
    "mamba_conv_state_bytes": (_i64, [_dp]),
    "mamba_decode_supported": (ctypes.c_int, [_dp]),
    "mamba_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mamba_conv_update": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mamba_state_update": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _vp,
                                          _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "mamba_spec_commit": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _vp, _vp]),
    "mamba_conv_varlen": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _vp, _vp]),
    "mamba1_conv_update": (ctypes.c_int, [_d1, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mamba1_state_update": (ctypes.c_int, [_d1, _vp, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                           _vp, _vp, _vp, _vp]),
    "mamba_slot_copy": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i32, _vp, _vp]),
    "mamba_int8_entry_bytes": (_sz, [_dp]),
    "mamba_ckpt_store_int8": (ctypes.c_int, [_dp, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _i64, _vp, _vp]),
    "mamba_ckpt_load_int8": (ctypes.c_int, [_dp, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _i64, _vp, _vp]),
    "mamba_chunk_scan_workspace_bytes": (_sz, [_dp, _i32, _i32, _i32]),
    "mamba_chunk_scan": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp, _vp]),
    "mamba_chunk_scan_noalloc": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32,
                                                _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp]),
    "mamba_chunk_scan_static_scratch_bytes": (_sz, []),
    "gdn_state_update": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                        _i32, _f32, _vp, _vp, _vp]),
    "gdn_state_update_int8": (ctypes.c_int, [_dp, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _f32,
                                             _vp, _vp, _vp]),
    "gdn_chunk_scan_workspace_bytes": (_sz, [_dp, _i32, _i32]),
    "gdn_chunk_scan": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _i32, _i32, _i32, _f32, _vp, _vp, _sz, _vp, _vp]),
    "la_state_update": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _f32, _vp, _vp,
                                       _i32, _i32, _f32, _vp, _vp, _vp]),
    "la_qk_norm_rope": (ctypes.c_int, [_dp, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _f32, _vp, _vp, _i32, _i32, _vp,
                                       _i64, _vp, _i64, _vp]),
    "la_chunk_scan_workspace_bytes": (_sz, [_dp, _i32, _i32]),
    "la_chunk_scan": (ctypes.c_int, [_dp, _vp, _i64, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _i64, _vp, _i64,
                                     _vp, _i64, _vp, _f32, _vp, _vp, _sz, _vp, _vp]),
    "mamba_batch_plan": (ctypes.c_int, [_vp, _vp, _i32, _vp, _i64, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp]),
    "mamba_check_slot_ids": (ctypes.c_int, [_vp, _i32, _vp, _i32, _i64, ctypes.POINTER(_i64)]),
    "mamba_selftest_wait_timeout": (ctypes.c_int, [_vp, _vp, _vp]),
}


def lib():
    """The loaded library; raises if it was not built (there is no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with recurrent_state_update_gb300.build.build()")
            h = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(h, name)
                f.restype = res
                f.argtypes = args
            _lib = h
        return _lib


def status_string(status: int) -> str:
    return lib().mamba_status_string(int(status)).decode()


def _check(rc: int, what: str):
    if rc != MAMBA_OK:
        raise MambaError(rc, what)


def _ptr(t):
    """Device pointer of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _cptr(t):
    if t is not None and not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return _ptr(t)


def _code_dtype(code):
    import torch
    return torch.bfloat16 if code == MAMBA_BF16 else torch.float32


def _expect(what, **tensors):
    """Raises ValueError when a tensor's dtype is not the one the call reads it as.  Each keyword
    is (tensor or None, the torch dtype the library expects)."""
    for name, (t, want) in tensors.items():
        if t is not None and t.dtype != want:
            raise ValueError(f"{what}: {name} must be {want}, got {t.dtype}")


def _layer_dtypes(desc):
    """(state, conv, activations, dt, fp32, int32, uint8) torch dtypes of a Mamba2 or Mamba1 desc."""
    import torch
    return (_code_dtype(desc.state_dtype), _code_dtype(desc.conv_dtype), _code_dtype(desc.act_dtype),
            _code_dtype(desc.dt_dtype), torch.float32, torch.int32, torch.uint8)


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


# ------------------------------------------------------------------------------------------
# sizes
# ------------------------------------------------------------------------------------------

def mamba_conv_dim(desc: LayerDesc) -> int:
    return lib().mamba_conv_dim(ctypes.byref(desc))


def mamba_ssm_state_bytes(desc: LayerDesc) -> int:
    return lib().mamba_ssm_state_bytes(ctypes.byref(desc))


def mamba_conv_state_bytes(desc: LayerDesc) -> int:
    return lib().mamba_conv_state_bytes(ctypes.byref(desc))


def mamba_decode_supported(desc: LayerDesc) -> int:
    return lib().mamba_decode_supported(ctypes.byref(desc))


def mamba_selftest_wait_timeout(err_word, elapsed_ns=None, stream=None):
    """Diagnostic: one bounded wait that runs out (err_word: device int32; elapsed_ns: device int64)."""
    _check(lib().mamba_selftest_wait_timeout(_ptr(err_word), _ptr(elapsed_ns), _stream(stream)),
           "mamba_selftest_wait_timeout")


def mamba_check_slot_ids(slot_ids, num_slots: int, scratch_slots=None) -> tuple[int, int]:
    """Host-side check of one call's slot ids (numpy int32 arrays: (batch,) and (batch, ntok)).
    Returns (status, index of the first offending entry or -1)."""
    import numpy as np
    ids = np.ascontiguousarray(slot_ids, dtype=np.int32)
    sc = None if scratch_slots is None else np.ascontiguousarray(scratch_slots, dtype=np.int32)
    ntok = 0 if sc is None else (sc.shape[1] if sc.ndim == 2 else 1)
    bad = _i64(-1)
    rc = lib().mamba_check_slot_ids(ids.ctypes.data if ids.size else None, int(ids.shape[0]),
                                    None if sc is None else sc.ctypes.data, int(ntok), int(num_slots),
                                    ctypes.byref(bad))
    return rc, int(bad.value)


def mamba_chunk_scan_workspace_bytes(desc: LayerDesc, total_tokens: int, nseq: int, chunk: int) -> int:
    return lib().mamba_chunk_scan_workspace_bytes(ctypes.byref(desc), total_tokens, nseq, chunk)


# ------------------------------------------------------------------------------------------
# decode
# ------------------------------------------------------------------------------------------

def mamba_conv_update(desc: LayerDesc, conv_pool, slot_ids, xbc_in, conv_w, xbc_out, *, conv_b=None,
                      err_word=None, stream=None):
    """Causal conv1d + SiLU over (batch, ntok, conv_dim) inputs, conv state updated in place."""
    _, cv, act, _, f32, i32, _ = _layer_dtypes(desc)
    _expect("mamba_conv_update", conv_pool=(conv_pool, cv), slot_ids=(slot_ids, i32), xbc_in=(xbc_in, act),
            conv_w=(conv_w, f32), xbc_out=(xbc_out, act), conv_b=(conv_b, f32), err_word=(err_word, i32))
    batch, ntok = int(slot_ids.shape[0]), int(xbc_in.shape[1])
    rc = lib().mamba_conv_update(ctypes.byref(desc), _ptr(conv_pool), conv_pool.stride(0), conv_pool.shape[0],
                                 _cptr(slot_ids), batch, ntok, _cptr(xbc_in), _cptr(conv_w), _cptr(conv_b),
                                 _cptr(xbc_out), _ptr(err_word), _stream(stream))
    _check(rc, "mamba_conv_update")


def mamba_state_update(desc: LayerDesc, ssm_pool, slot_ids, xbc, dt, A, y, *, conv_pool=None, conv_w=None,
                       conv_b=None, scratch_slots=None, D=None, dt_bias=None, dt_softplus=True, z=None,
                       err_word=None, stream=None):
    """The batched decode step (conv fused when ``conv_pool`` is given), in place on the pools."""
    st, cv, act, dtt, f32, i32, _ = _layer_dtypes(desc)
    _expect("mamba_state_update", ssm_pool=(ssm_pool, st), slot_ids=(slot_ids, i32), xbc=(xbc, act), dt=(dt, dtt),
            A=(A, f32), y=(y, act), conv_pool=(conv_pool, cv), conv_w=(conv_w, f32), conv_b=(conv_b, f32),
            scratch_slots=(scratch_slots, i32), D=(D, f32), dt_bias=(dt_bias, f32), z=(z, act),
            err_word=(err_word, i32))
    batch, ntok = int(slot_ids.shape[0]), int(xbc.shape[1])
    conv_stride = conv_pool.stride(0) if conv_pool is not None else 0
    rc = lib().mamba_state_update(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), ssm_pool.shape[0],
                                  _ptr(conv_pool), conv_stride, _cptr(conv_w), _cptr(conv_b), _cptr(slot_ids),
                                  _cptr(scratch_slots), batch, ntok, _cptr(xbc), _cptr(dt), _cptr(A), _cptr(D),
                                  _cptr(dt_bias), int(bool(dt_softplus)), _cptr(z), _cptr(y), _ptr(err_word),
                                  _stream(stream))
    _check(rc, "mamba_state_update")


def mamba_spec_commit(desc: LayerDesc, ssm_pool, slot_ids, scratch_slots, accept_len, *, conv_pool=None,
                      err_word=None, stream=None):
    """Keep accept_len[i] of the speculative tokens: copy the scratch state, re-seat the conv window."""
    st, cv, _, _, _, i32, _ = _layer_dtypes(desc)
    _expect("mamba_spec_commit", ssm_pool=(ssm_pool, st), slot_ids=(slot_ids, i32), scratch_slots=(scratch_slots, i32),
            accept_len=(accept_len, i32), conv_pool=(conv_pool, cv), err_word=(err_word, i32))
    batch, ntok = int(scratch_slots.shape[0]), int(scratch_slots.shape[1])
    conv_stride = conv_pool.stride(0) if conv_pool is not None else 0
    rc = lib().mamba_spec_commit(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), ssm_pool.shape[0],
                                 _ptr(conv_pool), conv_stride, _cptr(slot_ids), _cptr(scratch_slots),
                                 _cptr(accept_len), batch, ntok, _ptr(err_word), _stream(stream))
    _check(rc, "mamba_spec_commit")


# ------------------------------------------------------------------------------------------
# Mamba1 (S6) layers
# ------------------------------------------------------------------------------------------

def mamba1_conv_update(desc: Mamba1Desc, conv_pool, slot_ids, x_in, conv_w, x_out, *, conv_b=None, err_word=None,
                       stream=None):
    """Causal conv1d + SiLU of a Mamba1 layer over (batch, ntok, d_inner) inputs, conv state in place."""
    _, cv, act, _, f32, i32, _ = _layer_dtypes(desc)
    _expect("mamba1_conv_update", conv_pool=(conv_pool, cv), slot_ids=(slot_ids, i32), x_in=(x_in, act),
            conv_w=(conv_w, f32), x_out=(x_out, act), conv_b=(conv_b, f32), err_word=(err_word, i32))
    batch, ntok = int(slot_ids.shape[0]), int(x_in.shape[1])
    rc = lib().mamba1_conv_update(ctypes.byref(desc), _ptr(conv_pool), conv_pool.stride(0), conv_pool.shape[0],
                                  _cptr(slot_ids), batch, ntok, _cptr(x_in), _cptr(conv_w), _cptr(conv_b),
                                  _cptr(x_out), _ptr(err_word), _stream(stream))
    _check(rc, "mamba1_conv_update")


def mamba1_state_update(desc: Mamba1Desc, ssm_pool, slot_ids, x, dt, A, B, C, y, *, D=None, dt_bias=None,
                        dt_softplus=True, z=None, err_word=None, stream=None):
    """The batched single-token Mamba1 decode step, in place on the (slots, d_inner, d_state) pool."""
    st, _, act, dtt, f32, i32, _ = _layer_dtypes(desc)
    _expect("mamba1_state_update", ssm_pool=(ssm_pool, st), slot_ids=(slot_ids, i32), x=(x, act), dt=(dt, dtt),
            A=(A, f32), B=(B, act), C=(C, act), y=(y, act), D=(D, f32), dt_bias=(dt_bias, f32), z=(z, act),
            err_word=(err_word, i32))
    batch = int(slot_ids.shape[0])
    rc = lib().mamba1_state_update(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), ssm_pool.shape[0],
                                   _cptr(slot_ids), batch, _cptr(x), _cptr(dt), _cptr(A), _cptr(B), _cptr(C), _cptr(D),
                                   _cptr(dt_bias), int(bool(dt_softplus)), _cptr(z), _cptr(y), _ptr(err_word),
                                   _stream(stream))
    _check(rc, "mamba1_state_update")


# ------------------------------------------------------------------------------------------
# prefix-cache checkpoints
# ------------------------------------------------------------------------------------------

def mamba_slot_copy(desc: LayerDesc, ssm_pool, src_slots, dst_slots, *, conv_pool=None, err_word=None, stream=None):
    """Copy whole slot states src_slots[i] -> dst_slots[i] (checkpoint restore, copy-on-write)."""
    st, cv, _, _, _, i32, _ = _layer_dtypes(desc)
    _expect("mamba_slot_copy", ssm_pool=(ssm_pool, st), src_slots=(src_slots, i32), dst_slots=(dst_slots, i32),
            conv_pool=(conv_pool, cv), err_word=(err_word, i32))
    n = int(src_slots.shape[0])
    conv_stride = conv_pool.stride(0) if conv_pool is not None else 0
    rc = lib().mamba_slot_copy(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), ssm_pool.shape[0],
                               _ptr(conv_pool), conv_stride, _cptr(src_slots), _cptr(dst_slots), n, _ptr(err_word),
                               _stream(stream))
    _check(rc, "mamba_slot_copy")


def mamba_int8_entry_bytes(desc: LayerDesc) -> int:
    return lib().mamba_int8_entry_bytes(ctypes.byref(desc))


def mamba_ckpt_store_int8(desc: LayerDesc, ssm_pool, src_slots, dst_entries, store, *, conv_pool=None,
                          err_word=None, stream=None):
    """Quantise slots into int8 store entries (per-(head, d_state channel) symmetric scales)."""
    st, cv, _, _, _, i32, _ = _layer_dtypes(desc)
    _expect("mamba_ckpt_store_int8", ssm_pool=(ssm_pool, st), src_slots=(src_slots, i32),
            dst_entries=(dst_entries, i32), conv_pool=(conv_pool, cv), err_word=(err_word, i32))
    n = int(src_slots.shape[0])
    eb = mamba_int8_entry_bytes(desc)
    conv_stride = conv_pool.stride(0) if conv_pool is not None else 0
    rc = lib().mamba_ckpt_store_int8(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), _ptr(conv_pool),
                                     conv_stride, ssm_pool.shape[0], _cptr(src_slots), _cptr(dst_entries), n,
                                     _ptr(store), (store.numel() * store.element_size()) // eb, _ptr(err_word),
                                     _stream(stream))
    _check(rc, "mamba_ckpt_store_int8")


def mamba_ckpt_load_int8(desc: LayerDesc, ssm_pool, src_entries, dst_slots, store, *, conv_pool=None,
                         err_word=None, stream=None):
    """Dequantise int8 store entries into slots."""
    st, cv, _, _, _, i32, _ = _layer_dtypes(desc)
    _expect("mamba_ckpt_load_int8", ssm_pool=(ssm_pool, st), src_entries=(src_entries, i32),
            dst_slots=(dst_slots, i32), conv_pool=(conv_pool, cv), err_word=(err_word, i32))
    n = int(src_entries.shape[0])
    eb = mamba_int8_entry_bytes(desc)
    conv_stride = conv_pool.stride(0) if conv_pool is not None else 0
    rc = lib().mamba_ckpt_load_int8(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), _ptr(conv_pool),
                                    conv_stride, ssm_pool.shape[0], _cptr(src_entries), _cptr(dst_slots), n,
                                    _ptr(store), (store.numel() * store.element_size()) // eb, _ptr(err_word),
                                    _stream(stream))
    _check(rc, "mamba_ckpt_load_int8")


# ------------------------------------------------------------------------------------------
# prefill
# ------------------------------------------------------------------------------------------

def mamba_conv_varlen(desc: LayerDesc, cu_seqlens, xbc, conv_w, x_out, B_out, C_out, *, conv_pool=None,
                      slot_ids=None, has_initial_state=None, conv_b=None, err_word=None, stream=None):
    """Varlen causal conv1d + SiLU of a prefill batch into x | B | C, continuing each sequence
    from its conv state and writing the state back (when ``conv_pool`` is given)."""
    _, cv, act, _, f32, i32, u8 = _layer_dtypes(desc)
    _expect("mamba_conv_varlen", cu_seqlens=(cu_seqlens, i32), xbc=(xbc, act), conv_w=(conv_w, f32), x_out=(x_out, act),
            B_out=(B_out, act), C_out=(C_out, act), conv_pool=(conv_pool, cv), slot_ids=(slot_ids, i32),
            has_initial_state=(has_initial_state, u8), conv_b=(conv_b, f32), err_word=(err_word, i32))
    nseq = int(cu_seqlens.shape[0]) - 1
    total = int(xbc.shape[0])
    conv_stride = conv_pool.stride(0) if conv_pool is not None else 0
    num_slots = conv_pool.shape[0] if conv_pool is not None else 0
    rc = lib().mamba_conv_varlen(ctypes.byref(desc), _ptr(conv_pool), conv_stride, num_slots, _cptr(cu_seqlens),
                                 nseq, total, _cptr(slot_ids), _cptr(has_initial_state), _cptr(xbc), _cptr(conv_w),
                                 _cptr(conv_b), _cptr(x_out), _cptr(B_out), _cptr(C_out), _ptr(err_word),
                                 _stream(stream))
    _check(rc, "mamba_conv_varlen")


def mamba_chunk_scan(desc: LayerDesc, ssm_pool, cu_seqlens, slot_ids, x, dt, A, B, C, y, workspace, *,
                     has_initial_state=None, ckpt_slots=None, ckpt_interval=0, chunk=256, D=None, dt_bias=None,
                     dt_softplus=True, z=None, err_word=None, stream=None):
    """Varlen chunked prefill (SSD form); final states and checkpoints written into the pool."""
    st, _, act, dtt, f32, i32, u8 = _layer_dtypes(desc)
    _expect("mamba_chunk_scan", ssm_pool=(ssm_pool, st), cu_seqlens=(cu_seqlens, i32), slot_ids=(slot_ids, i32), x=(x, act),
            dt=(dt, dtt), A=(A, f32), B=(B, act), C=(C, act), y=(y, act), has_initial_state=(has_initial_state, u8),
            ckpt_slots=(ckpt_slots, i32), D=(D, f32), dt_bias=(dt_bias, f32), z=(z, act), err_word=(err_word, i32))
    nseq = int(cu_seqlens.shape[0]) - 1
    total = int(x.shape[0])
    max_ckpt = int(ckpt_slots.shape[1]) if ckpt_slots is not None else 0
    rc = lib().mamba_chunk_scan(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), ssm_pool.shape[0],
                                _cptr(cu_seqlens), nseq, total, _cptr(slot_ids), _cptr(has_initial_state),
                                _cptr(ckpt_slots), max_ckpt, int(ckpt_interval), int(chunk), _cptr(x), _cptr(dt),
                                _cptr(A), _cptr(B), _cptr(C), _cptr(D), _cptr(dt_bias), int(bool(dt_softplus)),
                                _cptr(z), _cptr(y), _ptr(workspace),
                                0 if workspace is None else workspace.numel() * workspace.element_size(),
                                _ptr(err_word), _stream(stream))
    _check(rc, "mamba_chunk_scan")


def mamba_chunk_scan_static_scratch_bytes() -> int:
    return lib().mamba_chunk_scan_static_scratch_bytes()


def mamba_chunk_scan_noalloc(desc: LayerDesc, ssm_pool, cu_seqlens, slot_ids, x, dt, A, B, C, y, *,
                             has_initial_state=None, ckpt_slots=None, ckpt_interval=0, chunk=256, D=None,
                             dt_bias=None, dt_softplus=True, z=None, err_word=None, stream=None):
    """mamba_chunk_scan for callers that cannot allocate: the library's fixed scratch is used
    instead of a caller workspace (see the C header for its size limit and sharing rules)."""
    st, _, act, dtt, f32, i32, u8 = _layer_dtypes(desc)
    _expect("mamba_chunk_scan_noalloc", ssm_pool=(ssm_pool, st), cu_seqlens=(cu_seqlens, i32), slot_ids=(slot_ids, i32), x=(x, act),
            dt=(dt, dtt), A=(A, f32), B=(B, act), C=(C, act), y=(y, act), has_initial_state=(has_initial_state, u8),
            ckpt_slots=(ckpt_slots, i32), D=(D, f32), dt_bias=(dt_bias, f32), z=(z, act), err_word=(err_word, i32))
    nseq = int(cu_seqlens.shape[0]) - 1
    total = int(x.shape[0])
    max_ckpt = int(ckpt_slots.shape[1]) if ckpt_slots is not None else 0
    rc = lib().mamba_chunk_scan_noalloc(ctypes.byref(desc), _ptr(ssm_pool), ssm_pool.stride(0), ssm_pool.shape[0],
                                        _cptr(cu_seqlens), nseq, total, _cptr(slot_ids), _cptr(has_initial_state),
                                        _cptr(ckpt_slots), max_ckpt, int(ckpt_interval), int(chunk), _cptr(x),
                                        _cptr(dt), _cptr(A), _cptr(B), _cptr(C), _cptr(D), _cptr(dt_bias),
                                        int(bool(dt_softplus)), _cptr(z), _cptr(y), _ptr(err_word), _stream(stream))
    _check(rc, "mamba_chunk_scan_noalloc")


# ------------------------------------------------------------------------------------------
# gated delta rule layers
# ------------------------------------------------------------------------------------------

_gdn_types = None  # torch dtypes by code, and the current stream's handle


def _gdn_setup():
    global _gdn_types
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    now = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _gdn_types = ({MAMBA_F32: torch.float32, MAMBA_BF16: torch.bfloat16}, torch.int32, torch.uint8, now)
    return _gdn_types


def _gdn_refuse(what, tensors):
    """Raises the ValueError of the first of (name, tensor or None, dtype, least elements or -1, contiguous)
    that breaks its line.  Called when a call's quick checks have found that one does."""
    for name, t, want, least, dense in tensors:
        if t is None:
            continue
        _expect(what, **{name: (t, want)})
        if not t.is_cuda:
            raise ValueError(f"{what}: {name}: expected a CUDA tensor")
        if dense and not t.is_contiguous():
            raise ValueError(f"{what}: {name}: expected a contiguous tensor")
        if t.numel() < least:
            raise ValueError(f"{what}: {name} needs {least} elements, got {t.numel()}")
    raise ValueError(f"{what}: bad arguments")


def _gdn_pointers(what, tensors):
    """Device pointers of (name, tensor or None, dtype, least elements, contiguous), each checked.  A decode
    step's kernel takes a few microseconds, so the checks of a good call are kept to attribute reads."""
    out = []
    for name, t, want, least, dense in tensors:
        if t is None:
            out.append(None)
            continue
        if t.dtype is not want or not t.is_cuda or (least > 0 and t.numel() < least) or (dense and not t.is_contiguous()):
            _gdn_refuse(what, tensors)
        out.append(t.data_ptr())
    return out


def _gdn_slots(what, pool, H, P, N):
    """(elements from slot to slot, slots) of a pool whose slots each hold a dense (H, P, N) state, in that shape
    or flat."""
    shape, strides = pool.shape, pool.stride()
    if shape != (shape[0], H, P, N) or strides != (strides[0], P * N, N, 1):
        one = pool.select(0, 0) if len(shape) > 1 and shape[0] else pool
        if len(shape) < 2 or not one.is_contiguous() or (shape[0] and one.numel() < H * P * N) or (
                len(shape) == 4 and shape[1:] != (H, P, N)):
            raise ValueError(f"{what}: ssm_pool: expected slots of dense ({H}, {P}, {N}) states, got shape {tuple(shape)} "
                             f"with strides {tuple(strides)}")
    return strides[0], shape[0]


def gdn_state_update(desc: LayerDesc, ssm_pool, slot_ids, xbc, dt, beta, A, y, *, scratch_slots=None, dt_bias=None,
                     dt_softplus=True, beta_sigmoid=True, qk_l2norm=True, scale=None, err_word=None, stream=None):
    """The gated delta rule's step over (batch, ntok, conv_dim) convolved channels v | k | q, in
    place on the pool (or into ``scratch_slots``).  ``scale`` defaults to d_state ** -0.5."""
    code, i32, _, now = _gdn_types or _gdn_setup()
    H, P, N = desc.nheads, desc.head_dim, desc.d_state
    act, dtt, f32 = code[desc.act_dtype], code[desc.dt_dtype], code[MAMBA_F32]
    batch, ntok = slot_ids.shape[0], xbc.shape[1]
    rows = batch * ntok
    pool, ids, scr, xp, dp, bp, ap, bias, yp, err = _gdn_pointers("gdn_state_update", (
        ("ssm_pool", ssm_pool, code[desc.state_dtype], -1, False), ("slot_ids", slot_ids, i32, -1, True),
        ("scratch_slots", scratch_slots, i32, rows, True), ("xbc", xbc, act, rows * (H * P + 2 * desc.n_groups * N), True),
        ("dt", dt, dtt, rows * H, True), ("beta", beta, dtt, rows * H, True), ("A", A, f32, H, True),
        ("dt_bias", dt_bias, f32, H, True), ("y", y, act, rows * H * P, True), ("err_word", err_word, i32, 1, False)))
    stride, slots = _gdn_slots("gdn_state_update", ssm_pool, H, P, N)
    rc = (_lib or lib()).gdn_state_update(ctypes.byref(desc), pool, stride, slots, ids, scr, batch, ntok, xp, dp, bp, ap,
                                          bias, 1 if dt_softplus else 0, 1 if beta_sigmoid else 0,
                                          1 if qk_l2norm else 0, N ** -0.5 if scale is None else scale, yp, err,
                                          now(ssm_pool.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "gdn_state_update")


def gdn_state_update_int8(desc: LayerDesc, store, entries, xbc, dt, beta, A, y, *, dt_bias=None, dt_softplus=True,
                          beta_sigmoid=True, qk_l2norm=True, scale=None, err_word=None, stream=None):
    """The gated delta rule's step of one token on int8 entries (the layout of mamba_ckpt_store_int8),
    read, updated and requantised in place.  ``scale`` defaults to d_state ** -0.5."""
    code, i32, u8, now = _gdn_types or _gdn_setup()
    H, P, N = desc.nheads, desc.head_dim, desc.d_state
    act, dtt, f32 = code[desc.act_dtype], code[desc.dt_dtype], code[MAMBA_F32]
    batch = entries.shape[0]
    sp, ids, xp, dp, bp, ap, bias, yp, err = _gdn_pointers("gdn_state_update_int8", (
        ("store", store, store.dtype, -1, True), ("entries", entries, i32, -1, True),
        ("xbc", xbc, act, batch * (H * P + 2 * desc.n_groups * N), True), ("dt", dt, dtt, batch * H, True),
        ("beta", beta, dtt, batch * H, True), ("A", A, f32, H, True), ("dt_bias", dt_bias, f32, H, True),
        ("y", y, act, batch * H * P, True), ("err_word", err_word, i32, 1, False)))
    h = _lib or lib()
    ref = ctypes.byref(desc)
    rc = h.gdn_state_update_int8(ref, sp, store.numel() * store.element_size() // (h.mamba_int8_entry_bytes(ref) or 1), ids,
                                 batch, xp, dp, bp, ap, bias, 1 if dt_softplus else 0, 1 if beta_sigmoid else 0,
                                 1 if qk_l2norm else 0, N ** -0.5 if scale is None else scale, yp, err,
                                 now(store.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "gdn_state_update_int8")


def gdn_chunk_scan_workspace_bytes(desc: LayerDesc, total_tokens: int, nseq: int) -> int:
    return lib().gdn_chunk_scan_workspace_bytes(ctypes.byref(desc), total_tokens, nseq)


def gdn_chunk_scan(desc: LayerDesc, ssm_pool, cu_seqlens, slot_ids, v, k, q, dt, beta, A, y, workspace, *,
                   has_initial_state=None, ckpt_slots=None, ckpt_interval=0, dt_bias=None, dt_softplus=True,
                   beta_sigmoid=True, qk_l2norm=True, scale=None, err_word=None, stream=None):
    """The gated delta rule over a varlen prefill batch; final states and checkpoints written into the
    pool.  ``scale`` defaults to d_state ** -0.5."""
    code, i32, u8, now = _gdn_types or _gdn_setup()
    H, P, N = desc.nheads, desc.head_dim, desc.d_state
    act, dtt, f32 = code[desc.act_dtype], code[desc.dt_dtype], code[MAMBA_F32]
    nseq, total, GN = cu_seqlens.shape[0] - 1, v.shape[0], desc.n_groups * N
    if ckpt_slots is not None and ckpt_slots.dim() != 2:
        raise ValueError("gdn_chunk_scan: ckpt_slots: expected (sequences, checkpoints)")
    max_ckpt = 0 if ckpt_slots is None else ckpt_slots.shape[1]
    pool, cu, ids, init, ckpt, vp, kp, qp, dp, bp, ap, bias, yp, wp, err = _gdn_pointers("gdn_chunk_scan", (
        ("ssm_pool", ssm_pool, code[desc.state_dtype], -1, False), ("cu_seqlens", cu_seqlens, i32, -1, True),
        ("slot_ids", slot_ids, i32, nseq, True), ("has_initial_state", has_initial_state, u8, nseq, True),
        ("ckpt_slots", ckpt_slots, i32, nseq * max_ckpt, True), ("v", v, act, total * H * P, True), ("k", k, act, total * GN, True),
        ("q", q, act, total * GN, True), ("dt", dt, dtt, total * H, True), ("beta", beta, dtt, total * H, True),
        ("A", A, f32, H, True), ("dt_bias", dt_bias, f32, H, True), ("y", y, act, total * H * P, True),
        ("workspace", workspace, workspace.dtype, -1, True), ("err_word", err_word, i32, 1, False)))
    stride, slots = _gdn_slots("gdn_chunk_scan", ssm_pool, H, P, N)
    rc = (_lib or lib()).gdn_chunk_scan(ctypes.byref(desc), pool, stride, slots, cu, nseq, total, ids, init, ckpt, max_ckpt,
                                        ckpt_interval, vp, kp, qp, dp, bp, ap, bias, 1 if dt_softplus else 0,
                                        1 if beta_sigmoid else 0, 1 if qk_l2norm else 0, N ** -0.5 if scale is None else scale, yp, wp,
                                        workspace.numel() * workspace.element_size(), err,
                                        now(ssm_pool.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "gdn_chunk_scan")


# ------------------------------------------------------------------------------------------
# linear attention layers
# ------------------------------------------------------------------------------------------

def _la_rows(what, name, t, tokens, heads, dim):
    """Elements from token to token of a (tokens, heads, dim) tensor whose tokens are each dense, in that shape or flat."""
    shape, strides = t.shape, t.stride()
    if shape == (tokens, heads, dim):
        dense = strides[2] == 1 and (strides[1] == dim or heads == 1)
    else:
        dense = shape == (tokens, heads * dim) and strides[1] == 1
    if not dense or (tokens > 1 and strides[0] < heads * dim):
        raise ValueError(f"{what}: {name}: expected ({tokens}, {heads}, {dim}) with dense tokens, got shape {tuple(shape)} "
                         f"with strides {tuple(strides)}")
    return strides[0] if tokens > 1 else heads * dim


def la_state_update(desc: LayerDesc, ssm_pool, slot_ids, xbc, log_decay, y, *, scratch_slots=None, qk_norm=False, k_weight=None,
                    q_weight=None, eps=1e-6, positions=None, inv_freq=None, interleaved=False, scale=None, err_word=None,
                    stream=None):
    """Linear attention's step over (batch, ntok, conv_dim) channels v | k | q, in place on the pool (or into
    ``scratch_slots``), with the norm (``qk_norm``) and the rotation (``inv_freq``, ``positions``) of its keys and
    queries.  ``scale`` defaults to d_state ** -0.5."""
    code, i32, _, now = _gdn_types or _gdn_setup()
    H, P, N = desc.nheads, desc.head_dim, desc.d_state
    act, f32 = code[desc.act_dtype], code[MAMBA_F32]
    batch, ntok = slot_ids.shape[0], xbc.shape[1]
    rows = batch * ntok
    rot = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    pool, ids, scr, xp, dp, kw, qw, pos, fp, yp, err = _gdn_pointers("la_state_update", (
        ("ssm_pool", ssm_pool, code[desc.state_dtype], -1, False), ("slot_ids", slot_ids, i32, -1, True),
        ("scratch_slots", scratch_slots, i32, rows, True), ("xbc", xbc, act, rows * (H * P + 2 * desc.n_groups * N), True),
        ("log_decay", log_decay, f32, H, True), ("k_weight", k_weight, f32, N, True), ("q_weight", q_weight, f32, N, True),
        ("positions", positions, i32, rows, True), ("inv_freq", inv_freq, f32, -1, True), ("y", y, act, rows * H * P, True),
        ("err_word", err_word, i32, 1, False)))
    stride, slots = _gdn_slots("la_state_update", ssm_pool, H, P, N)
    rc = (_lib or lib()).la_state_update(ctypes.byref(desc), pool, stride, slots, ids, scr, batch, ntok, xp, dp,
                                         1 if qk_norm else 0, kw, qw, eps, pos, fp, rot, 1 if interleaved else 0,
                                         N ** -0.5 if scale is None else scale, yp, err,
                                         now(ssm_pool.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "la_state_update")


def la_qk_norm_rope(desc: LayerDesc, k, q, k_out, q_out, *, qk_norm=True, k_weight=None, q_weight=None, eps=1e-6,
                    positions=None, inv_freq=None, interleaved=False, stream=None):
    """Norm and rotation of (tokens, n_groups, d_state) keys and queries, whose tokens may lie apart (views of a
    projection's rows); in place when ``k_out`` is ``k`` and ``q_out`` is ``q``.  Rows of a negative position are
    not written."""
    code, i32, _, now = _gdn_types or _gdn_setup()
    G, N = desc.n_groups, desc.d_state
    act, f32 = code[desc.act_dtype], code[MAMBA_F32]
    T = k.shape[0]
    rot = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    kp, qp, ko, qo, kw, qw, pos, fp = _gdn_pointers("la_qk_norm_rope", (
        ("k", k, act, -1, False), ("q", q, act, -1, False), ("k_out", k_out, act, -1, False), ("q_out", q_out, act, -1, False),
        ("k_weight", k_weight, f32, N, True), ("q_weight", q_weight, f32, N, True), ("positions", positions, i32, T, True),
        ("inv_freq", inv_freq, f32, -1, True)))
    ks, qs, kos, qos = [_la_rows("la_qk_norm_rope", n, t, T, G, N)
                        for n, t in (("k", k), ("q", q), ("k_out", k_out), ("q_out", q_out))]
    rc = (_lib or lib()).la_qk_norm_rope(ctypes.byref(desc), kp, ks, qp, qs, T, 1 if qk_norm else 0, kw, qw, eps, pos, fp, rot,
                                         1 if interleaved else 0, ko, kos, qo, qos,
                                         now(k.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "la_qk_norm_rope")


def la_chunk_scan_workspace_bytes(desc: LayerDesc, total_tokens: int, nseq: int) -> int:
    return lib().la_chunk_scan_workspace_bytes(ctypes.byref(desc), total_tokens, nseq)


def la_chunk_scan(desc: LayerDesc, ssm_pool, cu_seqlens, slot_ids, v, k, q, log_decay, y, workspace, *, has_initial_state=None,
                  ckpt_slots=None, ckpt_interval=0, scale=None, err_word=None, stream=None):
    """Linear attention over a varlen prefill batch; final states and checkpoints written into the pool.  The
    tokens of ``v``, ``k`` and ``q`` may lie apart (views of a projection's rows), and ``cu_seqlens`` may end before
    the last of them.  ``scale`` defaults to d_state ** -0.5."""
    code, i32, u8, now = _gdn_types or _gdn_setup()
    H, P, N, G = desc.nheads, desc.head_dim, desc.d_state, desc.n_groups
    act, f32 = code[desc.act_dtype], code[MAMBA_F32]
    nseq, total = cu_seqlens.shape[0] - 1, v.shape[0]
    if ckpt_slots is not None and ckpt_slots.dim() != 2:
        raise ValueError("la_chunk_scan: ckpt_slots: expected (sequences, checkpoints)")
    max_ckpt = 0 if ckpt_slots is None else ckpt_slots.shape[1]
    pool, cu, ids, init, ckpt, vp, kp, qp, dp, yp, wp, err = _gdn_pointers("la_chunk_scan", (
        ("ssm_pool", ssm_pool, code[desc.state_dtype], -1, False), ("cu_seqlens", cu_seqlens, i32, -1, True),
        ("slot_ids", slot_ids, i32, nseq, True), ("has_initial_state", has_initial_state, u8, nseq, True),
        ("ckpt_slots", ckpt_slots, i32, nseq * max_ckpt, True), ("v", v, act, -1, False), ("k", k, act, -1, False),
        ("q", q, act, -1, False), ("log_decay", log_decay, f32, H, True), ("y", y, act, total * H * P, True),
        ("workspace", workspace, workspace.dtype, -1, True), ("err_word", err_word, i32, 1, False)))
    stride, slots = _gdn_slots("la_chunk_scan", ssm_pool, H, P, N)
    vs = _la_rows("la_chunk_scan", "v", v, total, H, P)
    ks, qs = (_la_rows("la_chunk_scan", n, t, total, G, N) for n, t in (("k", k), ("q", q)))
    rc = (_lib or lib()).la_chunk_scan(ctypes.byref(desc), pool, stride, slots, cu, nseq, total, ids, init, ckpt, max_ckpt,
                                       ckpt_interval, vp, vs, kp, ks, qp, qs, dp, N ** -0.5 if scale is None else scale, yp, wp,
                                       workspace.numel() * workspace.element_size(), err,
                                       now(ssm_pool.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "la_chunk_scan")


# ------------------------------------------------------------------------------------------
# the plan of a batch
# ------------------------------------------------------------------------------------------

def mamba_batch_plan(new_tokens, computed, block_table, block: int, num_slots: int, *, cu_seqlens, slot_ids,
                     has_initial_state=None, copy_src=None, copy_dst=None, ckpt_slots=None, positions=None, token_rows=None,
                     err_word=None, stream=None):
    """The arguments of a batch's calls from its requests' lengths and block table, on the device, into the tensors
    given by keyword (each as long as the header says; ``positions`` and ``token_rows`` are as long as the most
    tokens of a batch)."""
    _, i32, u8, now = _gdn_types or _gdn_setup()
    rows = new_tokens.shape[0]
    for name, t, dims in (("block_table", block_table, 2), ("ckpt_slots", ckpt_slots, 2), ("positions", positions, 1),
                          ("token_rows", token_rows, 1)):
        if t is not None and t.dim() != dims:
            raise ValueError(f"mamba_batch_plan: {name}: expected {dims} dimension{'s' if dims > 1 else ''}")
    if block_table.shape[0] < rows or (rows and block_table.stride(1) != 1 and block_table.shape[1] > 1):
        raise ValueError("mamba_batch_plan: block_table: expected a row of dense pages for each request")
    per_token = [t.shape[0] for t in (positions, token_rows) if t is not None]
    max_tokens = min(per_token) if per_token else 2 ** 31 - 1
    if per_token and max(per_token) != max_tokens:
        raise ValueError("mamba_batch_plan: positions and token_rows: expected the same length")
    max_ckpt = 0 if ckpt_slots is None else ckpt_slots.shape[1]
    new, past, table, cu, ids, init, src, dst, ckpt, pos, tok, err = _gdn_pointers("mamba_batch_plan", (
        ("new_tokens", new_tokens, i32, -1, True), ("computed", computed, i32, rows, True), ("block_table", block_table, i32, -1, False),
        ("cu_seqlens", cu_seqlens, i32, rows + 1, True), ("slot_ids", slot_ids, i32, rows, True),
        ("has_initial_state", has_initial_state, u8, rows, True), ("copy_src", copy_src, i32, rows, True),
        ("copy_dst", copy_dst, i32, rows, True), ("ckpt_slots", ckpt_slots, i32, rows * max_ckpt, True),
        ("positions", positions, i32, -1, True), ("token_rows", token_rows, i32, -1, True), ("err_word", err_word, i32, 1, False)))
    cols = block_table.shape[1]
    rc = (_lib or lib()).mamba_batch_plan(new, past, rows, table, block_table.stride(0) if rows > 1 else cols, cols, block, num_slots,
                                          max_tokens, max_ckpt, cu, ids, init, src, dst, ckpt, pos, tok, err,
                                          now(new_tokens.device.index) if stream is None else stream.cuda_stream)
    if rc:
        _check(rc, "mamba_batch_plan")
