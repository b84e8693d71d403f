"""Python binding of liblachunked -- chunkwise-parallel causal linear attention on GB300.

Argument marshalling only: every step of the forward pass runs in the library's CUDA
kernels.  The functions named ``la_*`` mirror the C ABI in ``include/la_chunked.h`` one to
one (pointers are passed as integers).  ``chunked_fwd`` is a convenience wrapper taking
torch tensors; torch provides the device memory and the stream, nothing else.

There is no fallback: if ``liblachunked.so`` is missing or fails to load, every call
raises.  Build it with ``python -m chunkwise_causal_linear_gb300.build``.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblachunked.so")

LA_OK = 0
LA_ERR_NULL = -1
LA_ERR_SHAPE = -2
LA_ERR_UNSUPPORTED = -3
LA_ERR_WORKSPACE = -4
LA_ERR_CUDA = -5
LA_ERR_TIMEOUT = -6
LA_ERR_DEVICE = -7
LA_ERR_SCRATCH_LIMIT = -8
LA_ERR_ARG = -9

LA_FM_IDENTITY, LA_FM_ELU1, LA_FM_FAVOR = 0, 1, 2
LA_BF16, LA_F32 = 0, 1
LA_PATH_AUTO, LA_PATH_SIMT, LA_PATH_TC = 0, 1, 2

LA_GATE_VALUE, LA_GATE_LOG, LA_GATE_SIGMOID = 0, 1, 2
LA_RECURRENCE_CHUNK = 64
LA_ROTARY_HALF, LA_ROTARY_INTERLEAVED = 0, 1
LA_ROTARY_PLAIN, LA_ROTARY_LINEAR, LA_ROTARY_PARTS = 0, 1, 2
LA_ACT_NONE, LA_ACT_SILU, LA_ACT_SIGMOID = 0, 1, 2
LA_NORM_NONE, LA_NORM_RMS, LA_NORM_LAYER = 0, 1, 2

GATE_KINDS = {"value": LA_GATE_VALUE, "log": LA_GATE_LOG, "sigmoid": LA_GATE_SIGMOID}
ROTARY_LAYOUTS = {"half": LA_ROTARY_HALF, "interleaved": LA_ROTARY_INTERLEAVED}
ROTARY_SCALINGS = {"none": LA_ROTARY_PLAIN, "linear": LA_ROTARY_LINEAR, "parts": LA_ROTARY_PARTS}
ACTIVATIONS = {"none": LA_ACT_NONE, "silu": LA_ACT_SILU}
GATE_ACTIVATIONS = {**ACTIVATIONS, "sigmoid": LA_ACT_SIGMOID}
NORMS = {"none": LA_NORM_NONE, "rms": LA_NORM_RMS, "layer": LA_NORM_LAYER}
FEATURE_MAPS = {"identity": LA_FM_IDENTITY, "elu1": LA_FM_ELU1, "favor": LA_FM_FAVOR}

# every function the header declares (checked by the tests against include/la_chunked.h)
EXPORTS = ("la_chunked_fwd", "la_chunked_fwd_path", "la_chunked_fwd_host",
           "la_chunked_fwd_noalloc", "la_chunked_workspace_bytes", "la_chunked_plan",
           "la_last_device_status", "la_status_string", "la_cost_model", "la_decode_step",
           "la_decode_state_elems", "la_noncausal_fwd", "la_noncausal_workspace_bytes",
           "la_decay_fwd", "la_decay_decode_step", "la_decay_workspace_bytes", "la_decay_plan",
           "la_chunked_bwd", "la_chunked_bwd_workspace_bytes", "la_chunked_bwd_ll",
           "la_chunked_bwd_ll_workspace_bytes", "la_chunked_state",
           "la_state_combine", "la_chunked_fwd_init", "la_recurrence_fwd", "la_recurrence_bwd",
           "la_recurrence_step", "la_rotary_table", "la_rotary", "la_group_norm_fwd",
           "la_group_norm_bwd", "la_group_norm_bwd_workspace_bytes", "la_gated_fwd",
           "la_gated_workspace_bytes", "la_gated_bwd", "la_gated_bwd_workspace_bytes",
           "la_gated_step", "la_block_norm_fwd", "la_block_norm_bwd",
           "la_block_norm_bwd_workspace_bytes", "la_version")


class la_feature_map(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("m", ctypes.c_int), ("omega", ctypes.c_void_p)]


class la_plan_info(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("chunk", ctypes.c_int), ("n_chunks", ctypes.c_int),
                ("feature_dim", ctypes.c_int), ("grid_x", ctypes.c_int),
                ("grid_y", ctypes.c_int), ("block", ctypes.c_int),
                ("smem_bytes", ctypes.c_int), ("n_launches", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class la_strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_longlong), ("h", ctypes.c_longlong), ("l", ctypes.c_longlong)]


class LAError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {la_status_string(status)} ({status})" if what else
                         f"{la_status_string(status)} ({status})")


_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it is missing: there is no fallback path)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing; build it with "
                    "`python -m chunkwise_causal_linear_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            i, p, sz, ll = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong
            fmp = ctypes.POINTER(la_feature_map)
            common = [i, i, i, i, i, i, fmp, i, p, i, i, p, sz, p]
            L.la_chunked_fwd.argtypes = [p, p, p, p, *common]
            L.la_chunked_fwd.restype = i
            L.la_chunked_fwd_path.argtypes = [p, p, p, p, *common, i]
            L.la_chunked_fwd_path.restype = i
            L.la_chunked_fwd_host.argtypes = [p, p, p, p, p, p, p, p, *common]
            L.la_chunked_fwd_host.restype = i
            L.la_chunked_fwd_noalloc.argtypes = [p, p, p, p, i, i, i, i, i, i, fmp, i, p, i, i, p]
            L.la_chunked_fwd_noalloc.restype = i
            L.la_chunked_workspace_bytes.argtypes = [i, i, i, i, i, i, fmp, i, i, i]
            L.la_chunked_workspace_bytes.restype = sz
            L.la_chunked_plan.argtypes = [i, i, i, i, i, i, fmp, i, i, i, i, i, i,
                                          ctypes.POINTER(la_plan_info)]
            L.la_chunked_plan.restype = i
            L.la_last_device_status.argtypes = [p]
            L.la_last_device_status.restype = i
            L.la_status_string.argtypes = [i]
            L.la_status_string.restype = ctypes.c_char_p
            L.la_cost_model.argtypes = [ll, ll, ll, ctypes.POINTER(ll), ctypes.POINTER(ll)]
            L.la_cost_model.restype = i
            L.la_decode_step.argtypes = [p, p, p, p, p, p, i, i, i, i, fmp, i, p, i, ll, i, p]
            L.la_decode_step.restype = i
            L.la_decode_state_elems.argtypes = [i, i, i, i, fmp, i, ctypes.POINTER(ll)]
            L.la_decode_state_elems.restype = ll
            L.la_noncausal_fwd.argtypes = [p, p, p, p, i, i, i, i, i, fmp, i, i, p, sz, p]
            L.la_noncausal_fwd.restype = i
            L.la_noncausal_workspace_bytes.argtypes = [i, i, i, i, i, fmp, i, i]
            L.la_noncausal_workspace_bytes.restype = sz
            f = ctypes.c_float
            L.la_decay_fwd.argtypes = [p, p, p, p, i, i, i, i, i, i, fmp, i, f, i, p, sz, p, i]
            L.la_decay_fwd.restype = i
            L.la_decay_decode_step.argtypes = [p, p, p, p, p, p, i, i, i, i, fmp, i, f, i, p]
            L.la_decay_decode_step.restype = i
            L.la_decay_workspace_bytes.argtypes = [i, i, i, i, i, i, fmp, i, f, i]
            L.la_decay_workspace_bytes.restype = sz
            L.la_decay_plan.argtypes = [i, i, i, i, i, i, fmp, i, f, i, i, i,
                                        ctypes.POINTER(la_plan_info)]
            L.la_decay_plan.restype = i
            L.la_chunked_bwd.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, i, fmp, i, f, i, p, sz,
                                         p, i]
            L.la_chunked_bwd.restype = i
            L.la_chunked_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, fmp, i, i]
            L.la_chunked_bwd_workspace_bytes.restype = sz
            L.la_chunked_bwd_ll.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, i, fmp, i, p, i, i,
                                            p, sz, p, i]
            L.la_chunked_bwd_ll.restype = i
            L.la_chunked_bwd_ll_workspace_bytes.argtypes = [i, i, i, i, i, i, fmp, i, i, i]
            L.la_chunked_bwd_ll_workspace_bytes.restype = sz
            L.la_chunked_state.argtypes = [p, p, p, p, i, i, i, i, i, fmp, f, i, p]
            L.la_chunked_state.restype = i
            L.la_state_combine.argtypes = [p, p, p, p, i, i, i, i, f, p]
            L.la_state_combine.restype = i
            L.la_chunked_fwd_init.argtypes = [p, p, p, p, i, i, i, i, i, i, fmp, i, f, p, p, i, p, sz,
                                              p, i]
            L.la_chunked_fwd_init.restype = i
            stp, d8 = ctypes.POINTER(la_strides), ctypes.c_double
            L.la_recurrence_fwd.argtypes = [p] * 7 + [i] * 4 + [stp] * 3 + [i] * 4 + [p]
            L.la_recurrence_fwd.restype = i
            L.la_recurrence_bwd.argtypes = [p] * 9 + [i] * 4 + [stp] * 5 + [i] * 4 + [p]
            L.la_recurrence_bwd.restype = i
            L.la_recurrence_step.argtypes = [p] * 4 + [i] * 7 + [p]
            L.la_recurrence_step.restype = i
            L.la_rotary_table.argtypes = [i, d8, i, d8, d8, d8, d8, ctypes.POINTER(ctypes.c_ulonglong)]
            L.la_rotary_table.restype = i
            L.la_rotary.argtypes = [p] * 6 + [ll] + [i] * 6 + [stp] * 4 + [i, i, f, i, p]
            L.la_rotary.restype = i
            L.la_group_norm_fwd.argtypes = [p] * 5 + [i] * 4 + [stp] * 3 + [i, i, f, i, p]
            L.la_group_norm_fwd.restype = i
            L.la_group_norm_bwd.argtypes = [p] * 9 + [i] * 4 + [stp] * 5 + [i, i, f, i, p, sz, p]
            L.la_group_norm_bwd.restype = i
            L.la_group_norm_bwd_workspace_bytes.argtypes = [i] * 4
            L.la_group_norm_bwd_workspace_bytes.restype = sz
            L.la_gated_fwd.argtypes = [p] * 9 + [i] * 7 + [stp] * 5 + [f, i, p, sz, p, i]
            L.la_gated_fwd.restype = i
            L.la_gated_workspace_bytes.argtypes = [i] * 6
            L.la_gated_workspace_bytes.restype = sz
            L.la_gated_bwd.argtypes = [p] * 14 + [i] * 6 + [stp] * 8 + [f, i, p, sz, p, i]
            L.la_gated_bwd.restype = i
            L.la_gated_bwd_workspace_bytes.argtypes = [i] * 7
            L.la_gated_bwd_workspace_bytes.restype = sz
            L.la_gated_step.argtypes = [p] * 7 + [i] * 6 + [stp] * 4 + [f, i, p]
            L.la_gated_step.restype = i
            L.la_block_norm_fwd.argtypes = [p] * 9 + [i] * 3 + [stp] * 5 + [i] * 3 + [f] * 3 + [i, i, p]
            L.la_block_norm_fwd.restype = i
            L.la_block_norm_bwd.argtypes = [p] * 16 + [i] * 3 + [stp] * 8 + [i] * 3 + [f] * 3 + [i, i, p, sz, p]
            L.la_block_norm_bwd.restype = i
            L.la_block_norm_bwd_workspace_bytes.argtypes = [i] * 3
            L.la_block_norm_bwd_workspace_bytes.restype = sz
            L.la_version.argtypes = []
            L.la_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


def make_feature_map(kind="identity", m=0, omega_ptr=0) -> la_feature_map:
    if isinstance(kind, str):
        kind = FEATURE_MAPS[kind]
    return la_feature_map(int(kind), int(m), ctypes.c_void_p(int(omega_ptr) or None))


def _fm(fm):
    return None if fm is None else ctypes.byref(fm)


# ---- one-to-one wrappers of the C ABI ------------------------------------------------
def la_chunked_fwd(q, k, v, out, B, H, L, dk, dv, C, feature_map, normalize, level_weights,
                   num_levels, dtype, workspace, workspace_bytes, stream) -> int:
    return lib().la_chunked_fwd(q, k, v, out, B, H, L, dk, dv, C, _fm(feature_map), normalize,
                                level_weights, num_levels, dtype, workspace, workspace_bytes,
                                stream)


def la_chunked_fwd_path(q, k, v, out, B, H, L, dk, dv, C, feature_map, normalize,
                        level_weights, num_levels, dtype, workspace, workspace_bytes, stream,
                        path) -> int:
    return lib().la_chunked_fwd_path(q, k, v, out, B, H, L, dk, dv, C, _fm(feature_map),
                                     normalize, level_weights, num_levels, dtype, workspace,
                                     workspace_bytes, stream, path)


def la_chunked_fwd_host(q_host, k_host, v_host, out_host, q_dev, k_dev, v_dev, out_dev, B, H,
                        L, dk, dv, C, feature_map, normalize, level_weights, num_levels, dtype,
                        workspace, workspace_bytes, stream) -> int:
    return lib().la_chunked_fwd_host(q_host, k_host, v_host, out_host, q_dev, k_dev, v_dev,
                                     out_dev, B, H, L, dk, dv, C, _fm(feature_map), normalize,
                                     level_weights, num_levels, dtype, workspace,
                                     workspace_bytes, stream)


def la_chunked_fwd_noalloc(q, k, v, out, B, H, L, dk, dv, C, feature_map, normalize,
                           level_weights, num_levels, dtype, stream) -> int:
    """Forward pass that allocates nothing (for callers that cannot allocate device
    memory); scratch, where needed, comes from a fixed 8 MiB buffer inside the library.
    Calls that may overlap on the GPU must be serialised by the caller."""
    return lib().la_chunked_fwd_noalloc(q, k, v, out, B, H, L, dk, dv, C, _fm(feature_map),
                                        normalize, level_weights, num_levels, dtype, stream)


def la_chunked_workspace_bytes(B, H, L, dk, dv, C, feature_map, normalize, num_levels,
                               dtype) -> int:
    return lib().la_chunked_workspace_bytes(B, H, L, dk, dv, C, _fm(feature_map), normalize,
                                            num_levels, dtype)


def la_chunked_plan(B, H, L, dk, dv, C, feature_map, normalize, loglinear, num_levels, dtype,
                    path=LA_PATH_AUTO, num_sms=0):
    info = la_plan_info()
    rc = lib().la_chunked_plan(B, H, L, dk, dv, C, _fm(feature_map), normalize, loglinear,
                               num_levels, dtype, path, num_sms, ctypes.byref(info))
    return rc, info.as_dict()


def la_last_device_status(stream=0) -> int:
    return lib().la_last_device_status(stream)


def la_status_string(status: int) -> str:
    return lib().la_status_string(status).decode()


def la_cost_model(L, D, C):
    st, sc = ctypes.c_longlong(), ctypes.c_longlong()
    rc = lib().la_cost_model(L, D, C, ctypes.byref(st), ctypes.byref(sc))
    if rc != LA_OK:
        raise LAError(rc, "la_cost_model")
    return st.value, sc.value


def la_decode_step(q, k, v, out, state, zstate, B, H, dk, dv, feature_map, normalize,
                   level_weights, num_levels, t, dtype, stream) -> int:
    return lib().la_decode_step(q, k, v, out, state, zstate, B, H, dk, dv, _fm(feature_map),
                                normalize, level_weights, num_levels, t, dtype, stream)


def la_decode_state_elems(B, H, dk, dv, feature_map, num_levels):
    ze = ctypes.c_longlong()
    n = lib().la_decode_state_elems(B, H, dk, dv, _fm(feature_map), num_levels, ctypes.byref(ze))
    return n, ze.value


def la_noncausal_fwd(q, k, v, out, B, H, L, dk, dv, feature_map, normalize, dtype, workspace,
                     workspace_bytes, stream) -> int:
    return lib().la_noncausal_fwd(q, k, v, out, B, H, L, dk, dv, _fm(feature_map), normalize,
                                  dtype, workspace, workspace_bytes, stream)


def la_noncausal_workspace_bytes(B, H, L, dk, dv, feature_map, normalize, dtype) -> int:
    return lib().la_noncausal_workspace_bytes(B, H, L, dk, dv, _fm(feature_map), normalize, dtype)


def la_decay_fwd(q, k, v, out, B, H, L, dk, dv, C, feature_map, normalize, gamma, dtype,
                 workspace, workspace_bytes, stream, path) -> int:
    return lib().la_decay_fwd(q, k, v, out, B, H, L, dk, dv, C, _fm(feature_map), normalize,
                              gamma, dtype, workspace, workspace_bytes, stream, path)


def la_decay_decode_step(q, k, v, out, state, zstate, B, H, dk, dv, feature_map, normalize,
                         gamma, dtype, stream) -> int:
    return lib().la_decay_decode_step(q, k, v, out, state, zstate, B, H, dk, dv,
                                      _fm(feature_map), normalize, gamma, dtype, stream)


def la_decay_workspace_bytes(B, H, L, dk, dv, C, feature_map, normalize, gamma, dtype) -> int:
    return lib().la_decay_workspace_bytes(B, H, L, dk, dv, C, _fm(feature_map), normalize,
                                          gamma, dtype)


def la_decay_plan(B, H, L, dk, dv, C, feature_map, normalize, gamma, dtype, path, num_sms=0):
    info = la_plan_info()
    rc = lib().la_decay_plan(B, H, L, dk, dv, C, _fm(feature_map), normalize, gamma, dtype, path,
                             num_sms, ctypes.byref(info))
    return rc, info.as_dict()


def la_chunked_bwd(q, k, v, dout, dq, dk, dv, B, H, L, dk_, dv_, C, feature_map, normalize, gamma,
                   dtype, workspace, workspace_bytes, stream, path=LA_PATH_AUTO) -> int:
    return lib().la_chunked_bwd(q, k, v, dout, dq, dk, dv, B, H, L, dk_, dv_, C,
                                _fm(feature_map), normalize, gamma, dtype, workspace,
                                workspace_bytes, stream, path)


def la_chunked_bwd_ll(q, k, v, dout, dq, dk, dv, B, H, L, dk_, dv_, C, feature_map, normalize,
                      level_weights, num_levels, dtype, workspace, workspace_bytes, stream,
                      path=LA_PATH_AUTO) -> int:
    return lib().la_chunked_bwd_ll(q, k, v, dout, dq, dk, dv, B, H, L, dk_, dv_, C,
                                   _fm(feature_map), normalize, level_weights, num_levels, dtype,
                                   workspace, workspace_bytes, stream, path)


def la_chunked_bwd_ll_workspace_bytes(B, H, L, dk, dv, C, feature_map, normalize, num_levels,
                                      dtype) -> int:
    return lib().la_chunked_bwd_ll_workspace_bytes(B, H, L, dk, dv, C, _fm(feature_map),
                                                   normalize, num_levels, dtype)


def la_chunked_bwd_workspace_bytes(B, H, L, dk, dv, C, feature_map, normalize, dtype) -> int:
    return lib().la_chunked_bwd_workspace_bytes(B, H, L, dk, dv, C, _fm(feature_map), normalize,
                                                dtype)


def la_chunked_state(k, v, state, zstate, B, H, L, dk, dv, feature_map, gamma, dtype, stream) -> int:
    return lib().la_chunked_state(k, v, state, zstate, B, H, L, dk, dv, _fm(feature_map), gamma,
                                  dtype, stream)


def la_state_combine(state, zstate, seg_state, seg_zstate, B, H, D, dv, factor, stream) -> int:
    return lib().la_state_combine(state, zstate, seg_state, seg_zstate, B, H, D, dv, factor, stream)


def la_chunked_fwd_init(q, k, v, out, B, H, L, dk, dv, C, feature_map, normalize, gamma, state0,
                        zstate0, dtype, workspace, workspace_bytes, stream, path=LA_PATH_AUTO) -> int:
    return lib().la_chunked_fwd_init(q, k, v, out, B, H, L, dk, dv, C, _fm(feature_map), normalize,
                                     gamma, state0, zstate0, dtype, workspace, workspace_bytes,
                                     stream, path)


def la_recurrence_fwd(x, gate, h0, lengths, out, h_last, chunk_states, B, H, L, d, x_strides,
                      gate_strides, out_strides, gate_kind, complement, dtype, gate_dtype,
                      stream) -> int:
    return lib().la_recurrence_fwd(x, gate, h0, lengths, out, h_last, chunk_states, B, H, L, d,
                                   x_strides, gate_strides, out_strides, gate_kind, complement,
                                   dtype, gate_dtype, stream)


def la_recurrence_bwd(x, gate, chunk_states, lengths, dout, dh_last, dx, dgate, dh0, B, H, L, d,
                      x_strides, gate_strides, dout_strides, dx_strides, dgate_strides, gate_kind,
                      complement, dtype, gate_dtype, stream) -> int:
    return lib().la_recurrence_bwd(x, gate, chunk_states, lengths, dout, dh_last, dx, dgate, dh0,
                                   B, H, L, d, x_strides, gate_strides, dout_strides, dx_strides,
                                   dgate_strides, gate_kind, complement, dtype, gate_dtype, stream)


def la_recurrence_step(x, gate, state, out, B, H, d, gate_kind, complement, dtype, gate_dtype,
                       stream) -> int:
    return lib().la_recurrence_step(x, gate, state, out, B, H, d, gate_kind, complement, dtype,
                                    gate_dtype, stream)


def la_rotary_table(rot, base, scaling, factor, original_length, fast, slow, turns) -> int:
    return lib().la_rotary_table(rot, base, scaling, factor, original_length, fast, slow, turns)


def la_rotary(q, k, q_out, k_out, turns, positions, offset, B, H, Hk, L, d, rot, q_strides,
              k_strides, q_out_strides, k_out_strides, layout, inverse, amplitude, dtype,
              stream) -> int:
    return lib().la_rotary(q, k, q_out, k_out, turns, positions, offset, B, H, Hk, L, d, rot,
                           q_strides, k_strides, q_out_strides, k_out_strides, layout, inverse,
                           amplitude, dtype, stream)


def la_group_norm_fwd(x, weight, bias, gate, out, B, H, L, d, x_strides, gate_strides, out_strides,
                      center, activation, eps, dtype, stream) -> int:
    return lib().la_group_norm_fwd(x, weight, bias, gate, out, B, H, L, d, x_strides, gate_strides,
                                   out_strides, center, activation, eps, dtype, stream)


def la_group_norm_bwd(x, weight, bias, gate, dout, dx, dgate, dweight, dbias, B, H, L, d, x_strides,
                      gate_strides, dout_strides, dx_strides, dgate_strides, center, activation, eps,
                      dtype, workspace, workspace_bytes, stream) -> int:
    return lib().la_group_norm_bwd(x, weight, bias, gate, dout, dx, dgate, dweight, dbias, B, H, L,
                                   d, x_strides, gate_strides, dout_strides, dx_strides,
                                   dgate_strides, center, activation, eps, dtype, workspace,
                                   workspace_bytes, stream)


def la_group_norm_bwd_workspace_bytes(B, H, L, d) -> int:
    return lib().la_group_norm_bwd_workspace_bytes(B, H, L, d)


def la_gated_fwd(q, k, v, log_decay, state0, state, slots, lengths, out, B, H, Hk, L, dk, dv, n_slots,
                 q_strides, k_strides, v_strides, g_strides, out_strides, scale, dtype, workspace,
                 workspace_bytes, stream, path) -> int:
    return lib().la_gated_fwd(q, k, v, log_decay, state0, state, slots, lengths, out, B, H, Hk, L, dk, dv,
                              n_slots, q_strides, k_strides, v_strides, g_strides, out_strides, scale,
                              dtype, workspace, workspace_bytes, stream, path)


def la_gated_workspace_bytes(B, H, L, dk, dv, dtype) -> int:
    return lib().la_gated_workspace_bytes(B, H, L, dk, dv, dtype)


def la_gated_bwd(q, k, v, log_decay, state0, lengths, dout, dstate, grad_q, grad_k, grad_v, dlog_decay,
                 dlog_decay_head, dstate0, B, H, Hk, L, dk, dv, q_strides, k_strides, v_strides, g_strides,
                 dout_strides, dq_strides, dk_strides, dv_strides, scale, dtype, workspace,
                 workspace_bytes, stream, path) -> int:
    return lib().la_gated_bwd(q, k, v, log_decay, state0, lengths, dout, dstate, grad_q, grad_k, grad_v,
                              dlog_decay, dlog_decay_head, dstate0, B, H, Hk, L, dk, dv, q_strides,
                              k_strides, v_strides, g_strides, dout_strides, dq_strides, dk_strides,
                              dv_strides, scale, dtype, workspace, workspace_bytes, stream, path)


def la_gated_bwd_workspace_bytes(B, H, Hk, L, dk, dv, dtype) -> int:
    return lib().la_gated_bwd_workspace_bytes(B, H, Hk, L, dk, dv, dtype)


def la_gated_step(q, k, v, log_decay, state, slots, out, B, H, Hk, dk, dv, n_slots, q_strides, k_strides,
                  v_strides, g_strides, scale, dtype, stream) -> int:
    return lib().la_gated_step(q, k, v, log_decay, state, slots, out, B, H, Hk, dk, dv, n_slots, q_strides,
                               k_strides, v_strides, g_strides, scale, dtype, stream)


def la_block_norm_fwd(y, residual, gate, post_weight, post_bias, pre_weight, pre_bias, h, n, B, L, d, y_strides,
                      residual_strides, gate_strides, h_strides, n_strides, post_norm, pre_norm, activation,
                      residual_scale, branch_scale, eps, dtype, residual_dtype, stream) -> int:
    return lib().la_block_norm_fwd(y, residual, gate, post_weight, post_bias, pre_weight, pre_bias, h, n, B, L, d,
                                   y_strides, residual_strides, gate_strides, h_strides, n_strides, post_norm,
                                   pre_norm, activation, residual_scale, branch_scale, eps, dtype,
                                   residual_dtype, stream)


def la_block_norm_bwd(y, residual, gate, post_weight, post_bias, pre_weight, pre_bias, dh, dn, dresidual, dy, dgate,
                      dpost_weight, dpost_bias, dpre_weight, dpre_bias, B, L, d, y_strides, residual_strides,
                      gate_strides, dh_strides, dn_strides, dresidual_strides, dy_strides, dgate_strides, post_norm,
                      pre_norm, activation, residual_scale, branch_scale, eps, dtype, residual_dtype, workspace,
                      workspace_bytes, stream) -> int:
    return lib().la_block_norm_bwd(y, residual, gate, post_weight, post_bias, pre_weight, pre_bias, dh, dn, dresidual,
                                   dy, dgate, dpost_weight, dpost_bias, dpre_weight, dpre_bias, B, L, d, y_strides,
                                   residual_strides, gate_strides, dh_strides, dn_strides, dresidual_strides,
                                   dy_strides, dgate_strides, post_norm, pre_norm, activation, residual_scale,
                                   branch_scale, eps, dtype, residual_dtype, workspace, workspace_bytes, stream)


def la_block_norm_bwd_workspace_bytes(B, L, d) -> int:
    return lib().la_block_norm_bwd_workspace_bytes(B, L, d)


def la_version() -> str:
    return lib().la_version().decode()


# ---- torch-tensor convenience ----------------------------------------------------------
def noncausal_fwd(q, k, v, feature_map="identity", omega=None, normalize=False, out=None,
                  workspace=None, stream=None):
    """Bidirectional linear attention of CUDA tensors q,k [B,H,L,dk], v [B,H,L,dv]."""
    import torch
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dtype = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, L, dv), dtype=q.dtype, device=q.device)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    need = la_noncausal_workspace_bytes(B, H, L, dk, dv, fm, int(normalize), dtype)
    if need == 0:
        raise LAError(LA_ERR_UNSUPPORTED, "la_noncausal_workspace_bytes")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_noncausal_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, L, dk,
                          dv, fm, int(normalize), dtype, workspace.data_ptr(), need, stream)
    if rc != LA_OK:
        raise LAError(rc, "la_noncausal_fwd")
    return out


def decode_state(B, H, dk, dv, feature_map="identity", m=0, num_levels=0, normalize=False,
                 device="cuda"):
    """Zero decoding state (and normaliser state when normalize) for la_decode_step."""
    import torch
    fm = make_feature_map(feature_map, m, 1 if feature_map == "favor" else 0)
    n, nz = la_decode_state_elems(B, H, dk, dv, fm, num_levels)
    if n == 0:
        raise LAError(LA_ERR_SHAPE, "la_decode_state_elems")
    S = torch.zeros(n, dtype=torch.float32, device=device)
    z = torch.zeros(nz, dtype=torch.float32, device=device) if normalize else None
    return S, z


def decode_step(q, k, v, state, zstate=None, t=0, feature_map="identity", omega=None,
                normalize=False, level_weights=None, out=None, stream=None):
    """One decoding step: q, k [B,H,dk], v [B,H,dv] CUDA tensors (one token per head);
    state / zstate from decode_state(); level_weights [B,H,NL] fp32 for the log-linear
    mask, with t the token position.  Returns out [B,H,dv]."""
    import torch
    B, H, dk = q.shape
    dv = v.shape[-1]
    dtype = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    nl = level_weights.shape[-1] if level_weights is not None else 0
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                        state.data_ptr(), zstate.data_ptr() if zstate is not None else None,
                        B, H, dk, dv, fm, int(normalize),
                        level_weights.data_ptr() if level_weights is not None else None,
                        nl, int(t), dtype, stream)
    if rc != LA_OK:
        raise LAError(rc, "la_decode_step")
    return out



def decay_fwd(q, k, v, gamma, C=64, feature_map="identity", omega=None, normalize=False,
              out=None, workspace=None, stream=None, path=LA_PATH_AUTO):
    """Causal linear attention with the Retention decay gamma (la_decay_fwd) of CUDA
    tensors q,k [B,H,L,dk], v [B,H,L,dv]."""
    import torch
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors")
    dtype = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, L, dv), dtype=q.dtype, device=q.device)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    need = la_decay_workspace_bytes(B, H, L, dk, dv, C, fm, int(normalize), float(gamma), dtype)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_decay_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, L, dk, dv,
                      C, fm, int(normalize), float(gamma), dtype,
                      workspace.data_ptr() if need else None, need, stream, path)
    if rc != LA_OK:
        raise LAError(rc, "la_decay_fwd")
    return out


def decay_decode_step(q, k, v, state, gamma, zstate=None, feature_map="identity", omega=None,
                      normalize=False, out=None, stream=None):
    """One decoding step with the Retention decay (la_decay_decode_step); state / zstate
    from decode_state().  Returns out [B,H,dv]."""
    import torch
    B, H, dk = q.shape
    dv = v.shape[-1]
    dtype = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_decay_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              state.data_ptr(), zstate.data_ptr() if zstate is not None else None,
                              B, H, dk, dv, fm, int(normalize), float(gamma), dtype, stream)
    if rc != LA_OK:
        raise LAError(rc, "la_decay_decode_step")
    return out


def chunked_bwd(q, k, v, dout, C=64, feature_map="identity", omega=None, normalize=False,
                gamma=1.0, workspace=None, stream=None, path=LA_PATH_AUTO):
    """(dq, dk, dv) of the causal forward for CUDA tensors q,k [B,H,L,dk], v, dout [B,H,L,dv]."""
    import torch
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dtype = _dtype_code(q)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    need = la_chunked_bwd_workspace_bytes(B, H, L, dk, dv, C, fm, int(normalize), dtype)
    if need == 0:
        raise LAError(LA_ERR_UNSUPPORTED, "la_chunked_bwd_workspace_bytes")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dq, dk_t, dv_t = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_chunked_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                        dq.data_ptr(), dk_t.data_ptr(), dv_t.data_ptr(), B, H, L, dk, dv, C, fm,
                        int(normalize), float(gamma), dtype, workspace.data_ptr(), need, stream,
                        path)
    if rc != LA_OK:
        raise LAError(rc, "la_chunked_bwd")
    return dq, dk_t, dv_t


def chunked_bwd_ll(q, k, v, dout, level_weights, C=64, feature_map="identity", omega=None,
                   normalize=False, workspace=None, stream=None, path=LA_PATH_AUTO):
    """(dq, dk, dv) of the log-linear forward (level_weights [B,H,L,NL] fp32 CUDA tensor)."""
    import torch
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dtype = _dtype_code(q)
    nl = level_weights.shape[-1]
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    need = la_chunked_bwd_ll_workspace_bytes(B, H, L, dk, dv, C, fm, int(normalize), nl, dtype)
    if need == 0:
        raise LAError(LA_ERR_UNSUPPORTED, "la_chunked_bwd_ll_workspace_bytes")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    dq, dk_t, dv_t = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_chunked_bwd_ll(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                           dq.data_ptr(), dk_t.data_ptr(), dv_t.data_ptr(), B, H, L, dk, dv, C, fm,
                           int(normalize), level_weights.data_ptr(), nl, dtype,
                           workspace.data_ptr(), need, stream, path)
    if rc != LA_OK:
        raise LAError(rc, "la_chunked_bwd_ll")
    return dq, dk_t, dv_t


def chunked_state(k, v, feature_map="identity", omega=None, gamma=1.0, normalize=True,
                  stream=None):
    """(state [B,H,D,dv], zstate [B,H,D] or None) a causal pass over k, v ends with."""
    import torch
    B, H, L, dk = k.shape
    dv = v.shape[-1]
    D = omega.shape[0] if omega is not None else dk
    S = torch.empty((B, H, D, dv), dtype=torch.float32, device=k.device)
    z = torch.empty((B, H, D), dtype=torch.float32, device=k.device) if normalize else None
    fm = make_feature_map(feature_map, D if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    if stream is None:
        stream = torch.cuda.current_stream(k.device).cuda_stream
    rc = la_chunked_state(k.data_ptr(), v.data_ptr(), S.data_ptr(),
                          z.data_ptr() if z is not None else None, B, H, L, dk, dv, fm,
                          float(gamma), _dtype_code(k), stream)
    if rc != LA_OK:
        raise LAError(rc, "la_chunked_state")
    return S, z


def chunked_fwd_init(q, k, v, state0, zstate0=None, C=64, feature_map="identity", omega=None,
                     normalize=False, gamma=1.0, out=None, workspace=None, stream=None,
                     path=LA_PATH_AUTO):
    """The causal forward of q, k, v started from state0 [B,H,D,dv] (zstate0 [B,H,D])."""
    import torch
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    dtype = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, L, dv), dtype=q.dtype, device=q.device)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    if gamma == 1.0:
        need = la_chunked_workspace_bytes(B, H, L, dk, dv, C, fm, int(normalize), 0, dtype)
    else:
        need = la_decay_workspace_bytes(B, H, L, dk, dv, C, fm, int(normalize), float(gamma), dtype)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_chunked_fwd_init(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, L, dk,
                             dv, C, fm, int(normalize), float(gamma),
                             state0.data_ptr() if state0 is not None else None,
                             zstate0.data_ptr() if zstate0 is not None else None, dtype,
                             workspace.data_ptr() if need else None, need, stream, path)
    if rc != LA_OK:
        raise LAError(rc, "la_chunked_fwd_init")
    return out


_dtype_codes = {}


def _dtype_code(t):
    code = _dtype_codes.get(t.dtype)
    if code is None:
        import torch
        _dtype_codes.update({torch.bfloat16: LA_BF16, torch.float32: LA_F32})
        code = _dtype_codes.get(t.dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {t.dtype}")
    return code


_GENERIC_WARN_TOKENS = 1 << 20
_warned_shapes = set()


def _warn_if_generic(B, H, L, dk, dv, C, fm, normalize, nl, dtype, path):
    """The automatic path falls back to the generic CUDA-core kernel for shapes outside the
    tensor-core kernels' coverage; on large bf16 problems that is 100-1000x slower, so say so
    (once per shape) instead of staying silent."""
    if path != LA_PATH_AUTO or dtype != LA_BF16 or B * H * L < _GENERIC_WARN_TOKENS:
        return
    rc, info = la_chunked_plan(B, H, L, dk, dv, C, fm, normalize, int(nl > 0), nl, dtype,
                               LA_PATH_AUTO, 0)
    key = (B, H, L, dk, dv, C, fm.kind, fm.m, normalize, nl)
    if rc == LA_OK and info["path"] == LA_PATH_SIMT and key not in _warned_shapes:
        import warnings
        _warned_shapes.add(key)
        warnings.warn(f"la_chunked_fwd: B={B} H={H} L={L} dk={dk} dv={dv} C={C} runs on the generic "
                      "CUDA-core path (outside the tensor-core kernels' coverage, see "
                      "la_chunked_fwd_path in la_chunked.h); expect it to be 100-1000x slower",
                      RuntimeWarning, stacklevel=3)


def chunked_fwd(q, k, v, C=64, feature_map="identity", omega=None, normalize=False,
                level_weights=None, out=None, workspace=None, stream=None, path=LA_PATH_AUTO):
    """out[B,H,L,dv] = chunkwise causal linear attention of CUDA tensors q,k [B,H,L,dk],
    v [B,H,L,dv] (bf16 or fp32, contiguous).  omega: [m, dk] fp32 CUDA tensor for
    feature_map="favor".  level_weights: [B,H,L,NL] fp32 CUDA tensor for the log-linear
    mask.  out / workspace are allocated with torch when not given."""
    import torch
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors")
    dtype = _dtype_code(q)
    if out is None:
        out = torch.empty((B, H, L, dv), dtype=q.dtype, device=q.device)
    fm = make_feature_map(feature_map, omega.shape[0] if omega is not None else 0,
                          omega.data_ptr() if omega is not None else 0)
    nl = level_weights.shape[-1] if level_weights is not None else 0
    _warn_if_generic(B, H, L, dk, dv, C, fm, int(normalize), nl, dtype, path)
    need = la_chunked_workspace_bytes(B, H, L, dk, dv, C, fm, int(normalize), nl, dtype)
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device).cuda_stream
    rc = la_chunked_fwd_path(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, L,
                             dk, dv, C, fm, int(normalize),
                             level_weights.data_ptr() if level_weights is not None else None,
                             nl, dtype, workspace.data_ptr() if need else None,
                             need, stream, path)
    if rc != LA_OK:
        raise LAError(rc, "la_chunked_fwd")
    return out


# ---- around the attention: recurrence, rotary positions, group norm ---------------------
_binding = None


def _layer_binding():
    """The compiled binding of these operators (raises if it is missing)."""
    global _binding
    if _binding is None:
        import importlib

        import torch  # noqa: F401  (its libraries, which the binding links)
        lib()
        try:
            _binding = importlib.import_module("._layer", __package__)
        except ImportError as e:
            raise RuntimeError(f"{os.path.join(_HERE, '_layer.so')} is missing or does not load ({e}); "
                               "build it with `python -m chunkwise_causal_linear_gb300.build`") from e
    return _binding


def recurrence_fwd(x, gate, h0=None, gate_kind="sigmoid", complement=False, lengths=None,
                   save_chunks=False, out=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + w_t x_t (la_recurrence_fwd) of CUDA tensors
    x, gate [B,H,L,d] (bf16 or fp32 each, strided views allowed).  gate_kind: "value", "log" or
    "sigmoid"; complement: w = 1 - a instead of 1.  h0 [B,H,d] fp32: the state before row 0.
    lengths [B] int32: rows behind a sequence's end are 0 and keep the state.  Returns (out,
    h_last [B,H,d] fp32), with save_chunks also the chunk states that recurrence_bwd reads."""
    return (_binding or _layer_binding()).recurrence_fwd(x, gate, h0, GATE_KINDS[gate_kind], complement,
                                                      lengths, save_chunks, out, stream)


def recurrence_bwd(x, gate, chunk_states, dout, dh_last=None, gate_kind="sigmoid",
                   complement=False, lengths=None, dx=None, dgate=None, stream=None):
    """(dx, dgate, dh0) of recurrence_fwd(..., save_chunks=True) for dout [B,H,L,d] and dh_last
    [B,H,d] fp32 (None: zero); dh0 [B,H,d] fp32 is the gradient of h0."""
    return (_binding or _layer_binding()).recurrence_bwd(x, gate, chunk_states, dout, dh_last,
                                                      GATE_KINDS[gate_kind], complement, lengths, dx,
                                                      dgate, stream)


def recurrence_step(x, gate, state, gate_kind="sigmoid", complement=False, out=None, stream=None):
    """One decoding step of the recurrence: x, gate [B,H,d] (this token), state [B,H,d] fp32
    updated in place.  Returns out [B,H,d]."""
    return (_binding or _layer_binding()).recurrence_step(x, gate, state, GATE_KINDS[gate_kind],
                                                       complement, out, stream)


class RotaryTable:
    """Frequencies of rotary(): turns (int64 CUDA tensor [rot/2], a turn per position in units
    of 2^-64), rot channels, amplitude of the rotated pairs."""

    def __init__(self, turns, rot, amplitude=1.0):
        self.turns, self.rot, self.amplitude = turns, rot, amplitude


def rotary_table(rot, base=10000.0, scaling="none", factor=1.0, original_length=0.0, fast=32.0,
                 slow=1.0, amplitude=1.0, device="cuda"):
    """The table rotary() reads, made once (la_rotary_table).  scaling: "none", "linear" (every
    frequency / factor) or "parts" (only those of few turns over original_length)."""
    import torch
    host = (ctypes.c_ulonglong * (rot // 2))()
    rc = la_rotary_table(rot, float(base), ROTARY_SCALINGS[scaling], float(factor),
                         float(original_length), float(fast), float(slow), host)
    if rc != LA_OK:
        raise LAError(rc, "la_rotary_table")
    signed = [v - (1 << 64) if v >> 63 else v for v in host]
    return RotaryTable(torch.tensor(signed, dtype=torch.int64, device=device), rot, float(amplitude))


def rotary(q, k, table, positions=None, offset=0, layout="half", inverse=False, q_out=None,
           k_out=None, stream=None):
    """q [B,H,L,d] and k [B,Hk,L,d] (k may be None) turned by their positions (la_rotary):
    positions [B,L] int32, or offset + t.  Strided views are allowed on both sides, and q_out=q,
    k_out=k for in place (k_out only with k).  inverse turns back, which is also the gradient.  Returns
    (q_out, k_out)."""
    return (_binding or _layer_binding()).rotary(q, k, table.turns, table.rot, table.amplitude, positions,
                                              offset, ROTARY_LAYOUTS[layout], inverse, q_out, k_out,
                                              stream)


def group_norm_fwd(x, weight=None, bias=None, gate=None, eps=1e-5, activation="silu", center=True,
                   out=None, stream=None):
    """Group norm of x [B,H,L,d] over each head's channels (la_group_norm_fwd), channels last on
    the way out: y = xh weight + bias, out [B,L,H*d] = y act(gate) with gate [B,L,H*d], else
    act(y).  weight, bias: fp32, H*d values, or None; center=False leaves the mean in."""
    return (_binding or _layer_binding()).group_norm_fwd(x, weight, bias, gate, eps, ACTIVATIONS[activation],
                                                      center, out, stream)


def group_norm_bwd(x, dout, weight=None, bias=None, gate=None, eps=1e-5, activation="silu",
                   center=True, dx=None, dgate=None, workspace=None, stream=None):
    """(dx, dgate, dweight, dbias) of group_norm_fwd for dout [B,L,H*d]; None where the forward
    had None, and dgate is taken with gate only.  workspace: contiguous device memory of
    la_group_norm_bwd_workspace_bytes, allocated where it is None or smaller."""
    return (_binding or _layer_binding()).group_norm_bwd(x, dout, weight, bias, gate, eps,
                                                      ACTIVATIONS[activation], center, dx, dgate,
                                                      workspace, stream)


# ---- gated attention ----------------------------------------------------------------------
def gated_fwd(q, k, v, log_decay, scale=1.0, state0=None, lengths=None, slots=None, state=None, out=None,
              workspace=None, stream=None, path=LA_PATH_AUTO):
    """Causal linear attention with a decay per head, or per token and head (la_gated_fwd): S_t =
    exp(g_t) S_{t-1} + k_t v_t^T, out_t = scale q_t^T S_t, for CUDA tensors q [B,H,L,dk], k [B,Hk,L,dk],
    v [B,Hk,L,dv] (bf16 or fp32, strided views allowed; H / Hk heads share a key head) and log_decay fp32
    [H] or [B,H,L].  state0, state [B,H,dk,dv] fp32: the states before the first and behind the last
    row; with slots [B] int32 they are pools [n,H,dk,dv] in which sequence b's lies at slots[b] (the same
    tensor for both updates the pool in place).  lengths [B] int32: rows behind a sequence's end are not
    used.  Returns (out [B,H,L,dv], state); without slots a state is allocated where none is given."""
    return (_binding or _layer_binding()).gated_fwd(q, k, v, log_decay, scale, state0, lengths, slots, state,
                                                    out, workspace, stream, path)


def gated_bwd(q, k, v, log_decay, dout, scale=1.0, state0=None, lengths=None, dstate=None, dq=None, dk=None,
              dv=None, decay_grad=True, workspace=None, stream=None, path=LA_PATH_AUTO):
    """(dq, dk, dv, dlog_decay, dstate0) of gated_fwd for dout [B,H,L,dv] and dstate [B,H,dk,dv] fp32, the
    gradient of the state behind the last row (None: zero).  dlog_decay has log_decay's shape (None
    without decay_grad); dk and dv of a shared key head are the sums over its heads."""
    return (_binding or _layer_binding()).gated_bwd(q, k, v, log_decay, dout, scale, state0, lengths, dstate, dq,
                                                    dk, dv, decay_grad, workspace, stream, path)


def gated_step(q, k, v, log_decay, state, scale=1.0, slots=None, out=None, stream=None):
    """One decoding step of the gated attention: q [B,H,dk], k [B,Hk,dk], v [B,Hk,dv] (this token),
    log_decay fp32 [H] or [B,H], state [B,H,dk,dv] fp32, or with slots [B] int32 a pool [n,H,dk,dv],
    updated in place.  Returns out [B,H,dv]."""
    return (_binding or _layer_binding()).gated_step(q, k, v, log_decay, state, scale, slots, out, stream)


# ---- norms around a block -----------------------------------------------------------------
def block_norm_fwd(y, residual, gate=None, activation="silu", post_norm="rms", post_weight=None, post_bias=None,
                   pre_norm="rms", pre_weight=None, pre_bias=None, residual_scale=1.0, branch_scale=1.0, eps=1e-5,
                   h=None, n=None, stream=None):
    """(h, n) behind a block with the output y and before the next one (la_block_norm_fwd): h = residual_scale
    residual + branch_scale act(gate) (norm(y) post_weight + post_bias), n = norm(h) pre_weight + pre_bias, for
    CUDA tensors [B,L,d] (strided views allowed).  y and gate bf16 or fp32; residual of the same type or
    fp32.  post_norm: "none", "rms" or "layer"; pre_norm: "rms", "layer" or "none", which leaves n out (None).
    activation of the gate: "none", "silu" or "sigmoid".  weights and biases: fp32 [d] or None.  h=residual
    and n=y work in place."""
    return (_binding or _layer_binding()).block_norm_fwd(y, residual, gate, GATE_ACTIVATIONS[activation],
                                                         NORMS[post_norm], post_weight, post_bias, NORMS[pre_norm],
                                                         pre_weight, pre_bias, residual_scale, branch_scale, eps, h, n,
                                                         stream)


def block_norm_bwd(y, residual, dh, dn, gate=None, activation="silu", post_norm="rms", post_weight=None,
                   post_bias=None, pre_norm="rms", pre_weight=None, pre_bias=None, residual_scale=1.0,
                   branch_scale=1.0, eps=1e-5, dr=None, dy=None, dgate=None, workspace=None, stream=None):
    """Gradients of block_norm_fwd for dh (None: zero) and dn (None with pre_norm "none"), as a dict: dy, dr, and
    dgate, dpost_w, dpost_b, dpre_w, dpre_b (None where the forward had None).  workspace: contiguous
    device memory of la_block_norm_bwd_workspace_bytes, allocated where it is None or smaller."""
    return (_binding or _layer_binding()).block_norm_bwd(y, residual, dh, dn, gate, GATE_ACTIVATIONS[activation],
                                                         NORMS[post_norm], post_weight, post_bias, NORMS[pre_norm],
                                                         pre_weight, pre_bias, residual_scale, branch_scale, eps, dr,
                                                         dy, dgate, workspace, stream)
