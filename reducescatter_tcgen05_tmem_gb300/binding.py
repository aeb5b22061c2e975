"""ctypes binding of libflux_gb300.so: argument marshalling only.

Every function here has the name and the argument order of its C entry point
in ``include/flux_gb300.h``.  Pointer arguments accept torch tensors (their
``data_ptr()`` is passed), plain integers, or None for NULL; arrays of R
pointers accept a list of tensors.  ``stream`` defaults to torch's current
CUDA stream.  A non-OK status raises :class:`FluxError`.  No step of the
computation happens in Python, and there is no fallback: importing this module
raises if the compiled library is missing.
"""
from __future__ import annotations

import array
import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
# FLUX_CHECKED=1 in the environment loads the checked build (bounds checks in
# every kernel, see flux_checks_enabled in the header) instead of the regular one
CHECKED = os.environ.get("FLUX_CHECKED", "") not in ("", "0")
LIB_PATH = os.path.join(HERE, "libflux_gb300_checked.so" if CHECKED else "libflux_gb300.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m reducescatter_tcgen05_tmem_gb300.build` "
        "(the library has no CPU or Python fallback)")

_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------- constants
FLUX_OK = 0
FLUX_ERR_INVALID_ARG = 1
FLUX_ERR_UNSUPPORTED = 2
FLUX_ERR_WORKSPACE = 3
FLUX_ERR_CUDA = 4
FLUX_ERR_TIMEOUT = 5
FLUX_ERR_NO_DEVICE = 6

FLUX_F16 = 0
FLUX_BF16 = 1

FLUX_SCORE_SOFTMAX = 0
FLUX_SCORE_SIGMOID = 1

FLUX_OP_GEMM = 0
FLUX_OP_AG_GEMM = 1
FLUX_OP_GEMM_RS = 2
FLUX_OP_MOE_AG = 3
FLUX_OP_MOE_RS = 4
FLUX_OP_MLP = 5
FLUX_OP_MOE_LAYERS = 6
FLUX_OP_MOE_EP_AG = 7
FLUX_OP_MOE_EP_RS = 8
FLUX_OP_AG_GEMM_PUSH = 9

FLUX_MAX_RANKS = 16
FLUX_MAX_EXPERTS = 1024
FLUX_MAX_GROUPS = 32
FLUX_BLOCK_MAX_H = 16384
FLUX_W4_MAX_ROWS = 1024
FLUX_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024

WAIT_SITES = {1: "ready flag", 2: "smem slot free", 3: "smem slot full",
              4: "accumulator free", 5: "accumulator full", 6: "drain",
              7: "deterministic turn", 8: "staged rows", 9: "unit schedule",
              10: "cluster shape", 11: "grid barrier", 12: "cluster exchange", 13: "check"}


class flux_opts_t(ctypes.Structure):
    _fields_ = [("epoch", ctypes.c_uint32), ("reserved0", ctypes.c_uint32),
                ("timeout_ns", ctypes.c_uint64), ("num_ctas", ctypes.c_int32),
                ("group_n", ctypes.c_int32), ("tiles_per_group", ctypes.c_int32),
                ("deterministic_rs", ctypes.c_int32), ("moe_pull_gather", ctypes.c_int32),
                ("moe_stage_ctas", ctypes.c_int32), ("rs_tile", ctypes.c_int32),
                ("moe_l1_ranks", ctypes.c_int32), ("trace", ctypes.c_void_p),
                ("trace_words", ctypes.c_uint64), ("ag_push", ctypes.c_int32),
                ("debug_probe", ctypes.c_int32),
                ("moe_static_schedule", ctypes.c_int32), ("rs_group", ctypes.c_int32),
                ("acc_whole", ctypes.c_int32)]


class flux_device_report_t(ctypes.Structure):
    _fields_ = [("status", ctypes.c_uint32), ("where", ctypes.c_uint32),
                ("arg0", ctypes.c_uint32), ("arg1", ctypes.c_uint32)]


class FluxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = _lib.flux_status_string(status).decode()
        extra = ""
        if status == FLUX_ERR_CUDA:
            extra = f" (cudaError {_lib.flux_last_cuda_error()})"
        super().__init__(f"{what}: {name}{extra}")


_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_vpp = ctypes.POINTER(ctypes.c_void_p)
_f = ctypes.c_float
_rows = ctypes.c_char_p  # an array of pointers as the bytes of _row_ptrs
_opt = ctypes.POINTER(flux_opts_t)

_SIGS = {
    "flux_version": ([], ctypes.c_int),
    "flux_checks_enabled": ([], ctypes.c_int),
    "flux_opts_size": ([], _sz),
    "flux_status_string": ([_i], ctypes.c_char_p),
    "flux_last_cuda_error": ([], ctypes.c_int),
    "flux_workspace_size": ([_i, _i, _i, _i, _i], _sz),
    "flux_moe_workspace_size": ([_i, _i, _i, _i, _i, _i, _i], _sz),
    "flux_workspace_init": ([_vp, _sz, _vp], _i),
    "flux_get_status": ([_vp, _sz, _vp, ctypes.POINTER(flux_device_report_t)], _i),
    "flux_gemm": ([_i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _opt, _vp], _i),
    "flux_ag_gemm": ([_i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _vp, _vp, _sz, _opt, _vp], _i),
    "flux_gemm_rs": ([_i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _vp, _sz, _opt, _vp], _i),
    "flux_gemm_rs_noalloc": ([_i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _opt, _vp], _i),
    "flux_moe_topk_gate": ([_i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "flux_moe_route": ([_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "flux_moe_ag_grouped_gemm": ([_i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vpp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _sz, _opt, _vp], _i),
    "flux_moe_grouped_gemm_rs": ([_i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vp, _vp, _vp,
                                  _vp, _vpp, _vp, _sz, _opt, _vp], _i),
    "flux_mlp_ag_rs": ([_i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _vpp, _vpp, _vp, _vp, _sz, _opt, _vp], _i),
    "flux_moe_layers": ([_i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _vp, _vp, _vpp, _vpp, _vp,
                         _vp, _sz, _opt, _vp], _i),
    "flux_tune_ag_gemm": ([_i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _vp, _vp, _sz, _vp, _opt], _i),
    "flux_tune_gemm_rs": ([_i, _i, _i, _i, _i, _vpp, _vpp, _vpp, _vp, _sz, _vp, _opt], _i),
    "flux_tune_moe_layer0": ([_i, _i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vpp, _vp, _vp,
                              _vp, _vp, _vp, _vp, _sz, _vp, _opt], _i),
    "flux_tune_moe_layer1": ([_i, _i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vp, _vp, _vp,
                              _vp, _vpp, _vp, _sz, _vp, _opt], _i),
    "flux_launch_info": ([_i, _i, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)], _i),
    "flux_tune_clear": ([], None),
    "flux_tune_count": ([], _i),
    "flux_moe_ep_dispatch_gemm": ([_i, _i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vpp, _vp,
                                   _vp, _vp, _vp, _vp, _vp, _sz, _opt, _vp], _i),
    "flux_moe_ep_gemm_combine": ([_i, _i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vp, _vp,
                                  _vp, _vp, _vpp, _vp, _sz, _opt, _vp], _i),
    "flux_block_norm": ([_i, _i, _i, _i, _i, _i, _i, _f, _vpp, _vpp, _vp, _vp, _vp, _vp, _vpp, _vpp,
                         _vp, _vp, _vp], _i),
    "flux_block_norm_workspace_size": ([_i, _i, _i, _i], _sz),
    "flux_block_norm_bwd": ([_i, _i, _i, _i, _i, _i, _i, _vpp, _vpp, _vp, _vp, _vp, _vp, _vp, _vp,
                             _vpp, _vpp, _vpp, _vpp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "flux_moe_balance_loss": ([_i, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _sz, _vp], _i),
    "flux_moe_balance_workspace_size": ([_i, _i, _i, _i], _sz),
    "flux_moe_router_bwd": ([_i, _i, _i, _i, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                             _vp, _vp], _i),
    "flux_w4_weight_bytes": ([_i, _i, _i], _sz),
    "flux_w4_workspace_size": ([_i, _i, _i, _i], _sz),
    "flux_w4_quantize": ([_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "flux_w4_gemv": ([_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "flux_moe_w4_layer0": ([_i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "flux_moe_w4_layer1": ([_i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
    "flux_layer_norm": ([_i, _i, _i, _i, _f, _f, _rows, _rows, _vp, _vp, _vp, _rows, _rows, _vp, _vp, _vp], _i),
    "flux_layer_norm_workspace_size": ([_i, _i], _sz),
    "flux_layer_norm_bwd": ([_i, _i, _i, _i, _f, _rows, _vp, _vp, _vp, _vp, _rows, _rows, _rows, _rows, _vp, _vp, _vp,
                             _sz, _vp], _i),
    "flux_moe_group_gate": ([_i, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _vp, _vp], _i),
    "flux_moe_group_gate_bwd": ([_i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _i, _vp, _vp], _i),
    "flux_q8_quantize": ([_i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "flux_q8_workspace_size": ([_i, _i, _i], _sz),
    "flux_q8_gemm": ([_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

EXPORTED = tuple(_SIGS)
if _lib.flux_opts_size() != ctypes.sizeof(flux_opts_t):
    raise ImportError(f"flux_opts_t: the binding's copy ({ctypes.sizeof(flux_opts_t)} bytes) does not match "
                      f"{LIB_PATH} ({_lib.flux_opts_size()} bytes); rebuild the library")
_OPT_FIELDS = frozenset(name for name, _ in flux_opts_t._fields_)


# ---------------------------------------------------------------- marshalling
def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_PTRS = {}  # ctypes array types by length


def _ptrs(xs):
    n = len(xs)
    make = _PTRS.get(n) or _PTRS.setdefault(n, ctypes.c_void_p * n)
    if n == 1:
        return make(_ptr(xs[0]))
    return make.from_buffer(array.array("Q", [_ptr(x) or 0 for x in xs]))


def _optional_ptrs(xs):
    return None if xs is None else _ptrs(xs)


_PACK = {}  # struct packers by length


def _row_ptrs(R, xs):
    """The pointers of R row shards (or None) as bytes: half the time of a ctypes array."""
    if xs is None:
        return None
    n = len(xs)
    if n < R <= FLUX_MAX_RANKS:
        raise ValueError(f"{n} row shards for {R} ranks")
    pack = _PACK.get(n) or _PACK.setdefault(n, struct.Struct(f"{n}P").pack)
    if n == 1:
        return pack(_ptr(xs[0]) or 0)
    return pack(*[_ptr(x) or 0 for x in xs])


def _nbytes(t):
    return t.numel() * t.element_size()


_current_raw_stream = None


def _stream(stream):
    if stream is None:
        global _current_raw_stream
        if _current_raw_stream is None:
            import torch
            torch.cuda.current_stream()  # initialises CUDA
            device, raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
            # the handle alone (0.2 us); torch.cuda.current_stream() builds a Stream
            # object for it (3 us)
            _current_raw_stream = lambda: raw(device())  # noqa: E731
        return _current_raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _opts(opts):
    if opts is None:
        return None
    if isinstance(opts, dict):
        o = flux_opts_t()
        for k, v in opts.items():
            if k not in _OPT_FIELDS:
                raise KeyError(f"flux_opts_t has no field {k!r}")
            if k == "trace" and v is not None and not isinstance(v, int):
                # a tensor: its address, and its size unless given
                if "trace_words" not in opts:
                    o.trace_words = _nbytes(v) // 8
                v = v.data_ptr()
            setattr(o, k, v)
        opts = o
    return ctypes.byref(opts)


def _check(st, what):
    if st != FLUX_OK:
        raise FluxError(st, what)


def dtype_code(t) -> int:
    """FLUX_F16 / FLUX_BF16 for a torch dtype or tensor."""
    import torch
    dt = t.dtype if hasattr(t, "dtype") else t
    if dt == torch.float16:
        return FLUX_F16
    if dt == torch.bfloat16:
        return FLUX_BF16
    raise ValueError(f"unsupported dtype {dt}")


# ---------------------------------------------------------------- API (same names as the C ABI)
def flux_version() -> int:
    return _lib.flux_version()


def flux_checks_enabled() -> bool:
    return bool(_lib.flux_checks_enabled())


def flux_opts_size() -> int:
    return int(_lib.flux_opts_size())


def flux_status_string(status: int) -> str:
    return _lib.flux_status_string(status).decode()


def flux_workspace_size(op: int, R: int, M: int, N: int, K: int) -> int:
    return int(_lib.flux_workspace_size(op, R, M, N, K))


def flux_moe_workspace_size(op: int, R: int, T: int, H: int, F: int, E: int, topk: int) -> int:
    return int(_lib.flux_moe_workspace_size(op, R, T, H, F, E, topk))


def flux_workspace_init(workspace, stream=None) -> None:
    _check(_lib.flux_workspace_init(_ptr(workspace), _nbytes(workspace), _stream(stream)),
           "flux_workspace_init")


def flux_get_status(workspace, stream=None):
    """(status, report) after synchronising the stream; never raises for device errors."""
    rep = flux_device_report_t()
    st = _lib.flux_get_status(_ptr(workspace), _nbytes(workspace), _stream(stream), ctypes.byref(rep))
    if st in (FLUX_ERR_CUDA, FLUX_ERR_WORKSPACE):
        raise FluxError(st, "flux_get_status")
    return st, {"status": rep.status, "where": WAIT_SITES.get(rep.where, rep.where),
                "arg0": rep.arg0, "arg1": rep.arg1}


def flux_gemm(M, N, K, dtype, A, B, C, workspace, opts=None, stream=None) -> None:
    _check(_lib.flux_gemm(M, N, K, dtype, _ptr(A), _ptr(B), _ptr(C), _ptr(workspace),
                          _nbytes(workspace), _opts(opts), _stream(stream)), "flux_gemm")


def flux_ag_gemm(R, M, N, K, dtype, x_shards, w_shards, out, ready_flags, workspace,
                 opts=None, stream=None) -> None:
    _check(_lib.flux_ag_gemm(R, M, N, K, dtype, _ptrs(x_shards), _ptrs(w_shards), _ptrs(out),
                             _ptr(ready_flags), _ptr(workspace), _nbytes(workspace), _opts(opts),
                             _stream(stream)), "flux_ag_gemm")


def flux_gemm_rs(R, M, N, K, dtype, a_shards, b_shards, out, workspace, opts=None,
                 stream=None) -> None:
    _check(_lib.flux_gemm_rs(R, M, N, K, dtype, _ptrs(a_shards), _ptrs(b_shards), _ptrs(out),
                             _ptr(workspace), _nbytes(workspace), _opts(opts), _stream(stream)),
           "flux_gemm_rs")


def flux_gemm_rs_noalloc(R, M, N, K, dtype, a_shards, b_shards, out, opts=None,
                         stream=None) -> None:
    """flux_gemm_rs without a workspace: scratch lives in a fixed device array of
    the library (FLUX_NOALLOC_SCRATCH_BYTES), for callers that cannot allocate."""
    _check(_lib.flux_gemm_rs_noalloc(R, M, N, K, dtype, _ptrs(a_shards), _ptrs(b_shards),
                                     _ptrs(out), _opts(opts), _stream(stream)),
           "flux_gemm_rs_noalloc")


def flux_moe_topk_gate(T, E, topk, logits, topk_ids, topk_weights, stream=None) -> None:
    """Top-k expert ids and softmax gate weights from fp32 router scores."""
    _check(_lib.flux_moe_topk_gate(T, E, topk, _ptr(logits), _ptr(topk_ids), _ptr(topk_weights),
                                   _stream(stream)), "flux_moe_topk_gate")


def flux_moe_route(T, E, topk, topk_ids, counts, offsets, slot_to_row, row_to_slot,
                   workspace=None, stream=None) -> None:
    _check(_lib.flux_moe_route(T, E, topk, _ptr(topk_ids), _ptr(counts), _ptr(offsets),
                               _ptr(slot_to_row), _ptr(row_to_slot), _ptr(workspace),
                               0 if workspace is None else _nbytes(workspace), _stream(stream)),
           "flux_moe_route")


def flux_moe_ag_grouped_gemm(R, T, H, F, E, topk, dtype, x_shards, w1_shards, topk_ids, h_out,
                             counts, offsets, slot_to_row, row_to_slot, ready_flags, workspace,
                             opts=None, stream=None) -> None:
    _check(_lib.flux_moe_ag_grouped_gemm(
        R, T, H, F, E, topk, dtype, _ptrs(x_shards), _ptrs(w1_shards), _ptr(topk_ids),
        _ptrs(h_out), _ptr(counts), _ptr(offsets), _ptr(slot_to_row), _ptr(row_to_slot),
        _ptr(ready_flags), _ptr(workspace), _nbytes(workspace), _opts(opts), _stream(stream)),
        "flux_moe_ag_grouped_gemm")


def flux_moe_grouped_gemm_rs(R, T, H, F, E, topk, dtype, h_shards, w2_shards, topk_ids,
                             topk_weights, offsets, slot_to_row, row_to_slot, out, workspace,
                             opts=None, stream=None) -> None:
    _check(_lib.flux_moe_grouped_gemm_rs(
        R, T, H, F, E, topk, dtype, _ptrs(h_shards), _ptrs(w2_shards), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(offsets), _ptr(slot_to_row), _ptr(row_to_slot), _ptrs(out),
        _ptr(workspace), _nbytes(workspace), _opts(opts), _stream(stream)),
        "flux_moe_grouped_gemm_rs")


def flux_mlp_ag_rs(R, M, H, F, dtype, x_shards, w1_shards, h, w2_shards, out, ready_flags,
                   workspace, opts=None, stream=None) -> None:
    """The dense MLP in one call: h = AG-GEMM(X, W1), out = GEMM-RS(h, W2)."""
    _check(_lib.flux_mlp_ag_rs(R, M, H, F, dtype, _ptrs(x_shards), _ptrs(w1_shards), _ptrs(h),
                               _ptrs(w2_shards), _ptrs(out), _ptr(ready_flags), _ptr(workspace),
                               _nbytes(workspace), _opts(opts), _stream(stream)), "flux_mlp_ag_rs")


def flux_moe_layers(R, T, H, F, E, topk, dtype, x_shards, w1_shards, w2_shards, topk_ids,
                    topk_weights, h, out, ready_flags, workspace, opts=None, stream=None) -> None:
    """The MoE layer in one call: routing, layer0 into h, layer1 into out."""
    _check(_lib.flux_moe_layers(R, T, H, F, E, topk, dtype, _ptrs(x_shards), _ptrs(w1_shards),
                                _ptrs(w2_shards), _ptr(topk_ids), _ptr(topk_weights), _ptrs(h),
                                _ptrs(out), _ptr(ready_flags), _ptr(workspace), _nbytes(workspace),
                                _opts(opts), _stream(stream)), "flux_moe_layers")


def flux_moe_ep_dispatch_gemm(R, tp, T, H, F, E, topk, dtype, x_shards, w1_shards, topk_ids,
                              h_out, counts, offsets, slot_to_row, row_to_slot, ready_flags,
                              workspace, opts=None, stream=None) -> None:
    """MoE layer0 under an EP x TP split (tp ranks per expert group)."""
    _check(_lib.flux_moe_ep_dispatch_gemm(
        R, tp, T, H, F, E, topk, dtype, _ptrs(x_shards), _ptrs(w1_shards), _ptr(topk_ids),
        _ptrs(h_out), _ptr(counts), _ptr(offsets), _ptr(slot_to_row), _ptr(row_to_slot),
        _ptr(ready_flags), _ptr(workspace), _nbytes(workspace), _opts(opts), _stream(stream)),
        "flux_moe_ep_dispatch_gemm")


def flux_moe_ep_gemm_combine(R, tp, T, H, F, E, topk, dtype, h_shards, w2_shards, topk_ids,
                             topk_weights, offsets, slot_to_row, row_to_slot, out, workspace,
                             opts=None, stream=None) -> None:
    """MoE layer1 + top-k combine under an EP x TP split."""
    _check(_lib.flux_moe_ep_gemm_combine(
        R, tp, T, H, F, E, topk, dtype, _ptrs(h_shards), _ptrs(w2_shards), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(offsets), _ptr(slot_to_row), _ptr(row_to_slot), _ptrs(out),
        _ptr(workspace), _nbytes(workspace), _opts(opts), _stream(stream)),
        "flux_moe_ep_gemm_combine")


def flux_block_norm_workspace_size(T: int, H: int, gate_rows: int = 0, gate_cols: int = 0) -> int:
    return int(_lib.flux_block_norm_workspace_size(T, H, gate_rows, gate_cols))


def flux_block_norm(R, T, H, dtype, post_norm, gate_rows, gate_cols, eps, x_shards, y_shards, w_post, gate,
                    res_scale, w_pre, x_out, u_out, rstd_y=None, rstd_x=None, stream=None) -> None:
    """Post-norm, gate, residual and the next block's pre-norm in one pass."""
    _check(_lib.flux_block_norm(R, T, H, dtype, post_norm, gate_rows, gate_cols, eps, _optional_ptrs(x_shards),
                                _optional_ptrs(y_shards), _ptr(w_post), _ptr(gate), _ptr(res_scale), _ptr(w_pre),
                                _optional_ptrs(x_out), _optional_ptrs(u_out), _ptr(rstd_y), _ptr(rstd_x), _stream(stream)),
           "flux_block_norm")


def flux_block_norm_bwd(R, T, H, dtype, post_norm, gate_rows, gate_cols, x_shards, y_shards, w_post, gate,
                        res_scale, w_pre, rstd_y, rstd_x, dx_out, du, dx, dy, dw_post, dgate, dres_scale,
                        dw_pre, workspace, stream=None) -> None:
    """Gradients of flux_block_norm."""
    _check(_lib.flux_block_norm_bwd(
        R, T, H, dtype, post_norm, gate_rows, gate_cols, _optional_ptrs(x_shards), _optional_ptrs(y_shards), _ptr(w_post),
        _ptr(gate), _ptr(res_scale), _ptr(w_pre), _ptr(rstd_y), _ptr(rstd_x), _optional_ptrs(dx_out), _optional_ptrs(du),
        _optional_ptrs(dx), _optional_ptrs(dy), _ptr(dw_post), _ptr(dgate), _ptr(dres_scale), _ptr(dw_pre), _ptr(workspace),
        _nbytes(workspace), _stream(stream)), "flux_block_norm_bwd")


def flux_moe_balance_workspace_size(T: int, E: int, topk: int, seqs: int) -> int:
    return int(_lib.flux_moe_balance_workspace_size(T, E, topk, seqs))


def flux_moe_balance_loss(T, E, topk, seqs, balance_coef, z_coef, logits, topk_ids, token_mask, loss, counts,
                          probs, tokens, lse, workspace, stream=None) -> None:
    """Balance and z losses of the router, with the per-expert counts."""
    _check(_lib.flux_moe_balance_loss(
        T, E, topk, seqs, balance_coef, z_coef, _ptr(logits), _ptr(topk_ids), _ptr(token_mask), _ptr(loss),
        _ptr(counts), _ptr(probs), _ptr(tokens), _ptr(lse), _ptr(workspace), _nbytes(workspace),
        _stream(stream)), "flux_moe_balance_loss")


def flux_moe_router_bwd(T, E, topk, seqs, balance_coef, z_coef, logits, topk_ids, topk_weights, token_mask, lse,
                        counts, tokens, dloss, dweights, dlogits, stream=None) -> None:
    """Gradient of the router scores from both losses and from the gate weights."""
    _check(_lib.flux_moe_router_bwd(
        T, E, topk, seqs, balance_coef, z_coef, _ptr(logits), _ptr(topk_ids), _ptr(topk_weights),
        _ptr(token_mask), _ptr(lse), _ptr(counts), _ptr(tokens), _ptr(dloss), _ptr(dweights), _ptr(dlogits),
        _stream(stream)), "flux_moe_router_bwd")


def flux_w4_weight_bytes(E: int, K: int, N: int) -> int:
    return int(_lib.flux_w4_weight_bytes(E, K, N))


def flux_w4_workspace_size(rows: int, N: int, K: int, E: int = 1) -> int:
    return int(_lib.flux_w4_workspace_size(rows, N, K, E))


def flux_w4_quantize(E, K, N, group, dtype, w, q, scales, stream=None) -> None:
    """4-bit codes and group scales of 16-bit weights [E x K x N]."""
    _check(_lib.flux_w4_quantize(E, K, N, group, dtype, _ptr(w), _ptr(q), _ptr(scales), _stream(stream)),
           "flux_w4_quantize")


def flux_w4_gemv(M, N, K, group, dtype, x, q, scales, out, workspace, stream=None) -> None:
    """out = x . W for few rows of x and 4-bit W."""
    _check(_lib.flux_w4_gemv(M, N, K, group, dtype, _ptr(x), _ptr(q), _ptr(scales), _ptr(out),
                             _ptr(workspace), _nbytes(workspace), _stream(stream)), "flux_w4_gemv")


def flux_moe_w4_layer0(T, H, F, E, topk, group, dtype, x, q1, scales1, topk_ids, h, workspace,
                       stream=None) -> None:
    """MoE layer0 of few tokens with 4-bit experts; h in slot order."""
    _check(_lib.flux_moe_w4_layer0(T, H, F, E, topk, group, dtype, _ptr(x), _ptr(q1), _ptr(scales1),
                                   _ptr(topk_ids), _ptr(h), _ptr(workspace), _nbytes(workspace),
                                   _stream(stream)), "flux_moe_w4_layer0")


def flux_moe_w4_layer1(T, H, F, E, topk, group, dtype, h, q2, scales2, topk_ids, topk_weights, out, workspace,
                       stream=None) -> None:
    """MoE layer1 + gate-weighted combine of few tokens with 4-bit experts."""
    _check(_lib.flux_moe_w4_layer1(T, H, F, E, topk, group, dtype, _ptr(h), _ptr(q2), _ptr(scales2),
                                   _ptr(topk_ids), _ptr(topk_weights), _ptr(out), _ptr(workspace),
                                   _nbytes(workspace), _stream(stream)), "flux_moe_w4_layer1")


def flux_layer_norm_workspace_size(T: int, H: int) -> int:
    return int(_lib.flux_layer_norm_workspace_size(T, H))


def flux_layer_norm(R, T, H, dtype, p, eps, x_shards, y_shards, rng, weight, bias, x_out, u_out, mean=None, rstd=None,
                    stream=None) -> None:
    """Dropout, residual and the next block's layer norm in one pass."""
    _check(_lib.flux_layer_norm(R, T, H, dtype, p, eps, _row_ptrs(R, x_shards), _row_ptrs(R, y_shards), _ptr(rng),
                                _ptr(weight), _ptr(bias), _row_ptrs(R, x_out), _row_ptrs(R, u_out), _ptr(mean),
                                _ptr(rstd), _stream(stream)), "flux_layer_norm")


def flux_layer_norm_bwd(R, T, H, dtype, p, x_out, rng, weight, mean, rstd, dx_out, du, dx, dy, dweight, dbias,
                        workspace, stream=None) -> None:
    """Gradients of flux_layer_norm."""
    _check(_lib.flux_layer_norm_bwd(
        R, T, H, dtype, p, _row_ptrs(R, x_out), _ptr(rng), _ptr(weight), _ptr(mean), _ptr(rstd), _row_ptrs(R, dx_out),
        _row_ptrs(R, du), _row_ptrs(R, dx), _row_ptrs(R, dy), _ptr(dweight), _ptr(dbias), _ptr(workspace),
        _nbytes(workspace), _stream(stream)), "flux_layer_norm_bwd")


def flux_moe_group_gate(T, E, topk, score, groups, topk_groups, group_top, renorm, scale, logits, bias, topk_ids,
                        topk_weights, stream=None) -> None:
    """Expert ids and weights of routing with groups."""
    _check(_lib.flux_moe_group_gate(T, E, topk, score, groups, topk_groups, group_top, renorm, scale, _ptr(logits),
                                    _ptr(bias), _ptr(topk_ids), _ptr(topk_weights), _stream(stream)),
           "flux_moe_group_gate")


def flux_moe_group_gate_bwd(T, E, topk, score, renorm, scale, logits, topk_ids, dweights, accumulate, dlogits,
                            stream=None) -> None:
    """Gradient of the logits from the gradient of flux_moe_group_gate's weights."""
    _check(_lib.flux_moe_group_gate_bwd(T, E, topk, score, renorm, scale, _ptr(logits), _ptr(topk_ids), _ptr(dweights),
                                        accumulate, _ptr(dlogits), _stream(stream)), "flux_moe_group_gate_bwd")


def flux_q8_quantize(rows, K, dtype, x, q, scales, stream=None) -> None:
    """8-bit codes and a scale for each row of 16-bit numbers."""
    _check(_lib.flux_q8_quantize(rows, K, dtype, _ptr(x), _ptr(q), _ptr(scales), _stream(stream)), "flux_q8_quantize")


def flux_q8_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.flux_q8_workspace_size(M, N, K))


def flux_q8_gemm(M, N, K, dtype, x, x_scales, w, w_scales, bias, out, workspace, stream=None) -> None:
    """out = x . w^T of 8-bit codes, times the rows' and the channels' scales."""
    _check(_lib.flux_q8_gemm(M, N, K, dtype, _ptr(x), _ptr(x_scales), _ptr(w), _ptr(w_scales), _ptr(bias), _ptr(out),
                             _ptr(workspace), _nbytes(workspace), _stream(stream)), "flux_q8_gemm")


def _tuned(st, what, best):
    _check(st, what)
    return {f: getattr(best, f) for f, _ in flux_opts_t._fields_}


def flux_tune_ag_gemm(R, M, N, K, dtype, x_shards, w_shards, out, ready_flags, workspace,
                      stream=None) -> dict:
    """Time the AllGather + GEMM candidates; record and return the fastest options."""
    best = flux_opts_t()
    return _tuned(_lib.flux_tune_ag_gemm(R, M, N, K, dtype, _ptrs(x_shards), _ptrs(w_shards),
                                         _ptrs(out), _ptr(ready_flags), _ptr(workspace),
                                         _nbytes(workspace), _stream(stream), ctypes.byref(best)),
                  "flux_tune_ag_gemm", best)


def flux_tune_gemm_rs(R, M, N, K, dtype, a_shards, b_shards, out, workspace, stream=None) -> dict:
    """Time the GEMM + ReduceScatter candidates; record and return the fastest options."""
    best = flux_opts_t()
    return _tuned(_lib.flux_tune_gemm_rs(R, M, N, K, dtype, _ptrs(a_shards), _ptrs(b_shards),
                                         _ptrs(out), _ptr(workspace), _nbytes(workspace),
                                         _stream(stream), ctypes.byref(best)),
                  "flux_tune_gemm_rs", best)


def flux_tune_moe_layer0(R, tp, T, H, F, E, topk, dtype, x_shards, w1_shards, topk_ids, h_out,
                         counts, offsets, slot_to_row, row_to_slot, ready_flags, workspace,
                         stream=None) -> dict:
    """Time the MoE layer0 candidates (staged / pull); record and return the fastest."""
    best = flux_opts_t()
    return _tuned(_lib.flux_tune_moe_layer0(
        R, tp, T, H, F, E, topk, dtype, _ptrs(x_shards), _ptrs(w1_shards), _ptr(topk_ids),
        _ptrs(h_out), _ptr(counts), _ptr(offsets), _ptr(slot_to_row), _ptr(row_to_slot),
        _ptr(ready_flags), _ptr(workspace), _nbytes(workspace), _stream(stream),
        ctypes.byref(best)), "flux_tune_moe_layer0", best)


def flux_tune_moe_layer1(R, tp, T, H, F, E, topk, dtype, h_shards, w2_shards, topk_ids,
                         topk_weights, offsets, slot_to_row, row_to_slot, out, workspace,
                         stream=None) -> dict:
    """Time the MoE layer1 candidates; record and return the fastest."""
    best = flux_opts_t()
    return _tuned(_lib.flux_tune_moe_layer1(
        R, tp, T, H, F, E, topk, dtype, _ptrs(h_shards), _ptrs(w2_shards), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(offsets), _ptr(slot_to_row), _ptr(row_to_slot), _ptrs(out),
        _ptr(workspace), _nbytes(workspace), _stream(stream), ctypes.byref(best)),
        "flux_tune_moe_layer1", best)


def flux_tune_clear() -> None:
    _lib.flux_tune_clear()


def flux_tune_count() -> int:
    return _lib.flux_tune_count()


def flux_launch_info(op, dtype) -> dict:
    """CTAs per cluster and resident CTAs of a dense op's kernel on this GPU."""
    cl, res = ctypes.c_int(0), ctypes.c_int(0)
    _check(_lib.flux_launch_info(op, dtype, ctypes.byref(cl), ctypes.byref(res)), "flux_launch_info")
    return {"cluster_ctas": cl.value, "resident_ctas": res.value}
