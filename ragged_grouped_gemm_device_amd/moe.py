"""ctypes binding of libmoe.so: the C ABI of include/moe.h with the same names.

Argument marshalling only: every step runs in the library's HIP kernels, on
torch's current HIP stream. torch tensors supply device memory; bf16 tensors
are passed by address (torch.bfloat16 or int16/uint16 bit patterns).
Failing to load the library raises immediately -- there is no fallback.
"""
from __future__ import annotations

import copy
import ctypes as C
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_LAUNCH = -4
MOE_ALIGN = 128
MOE_MX_BLOCK = 32
MOE_GLU_INTERLEAVE = 32
MOE_MAX_EXPERTS = 1024
MOE_MAX_ROWS = 1 << 30
MOE_ACT_SWIGLU = 0
MOE_ACT_GEGLU = 1
MOE_ACT_SRELU = 2   # non-gated relu(h)^2: FC1 width n
MOE_ACT_NONE = 3    # the dense linear layer's further activations
MOE_ACT_SILU = 4
MOE_ACT_GELU = 5
MOE_LINEAR_FWD = 0x1
MOE_LINEAR_BWD = 0x2
MOE_STAGE_FC1 = 0x01
MOE_STAGE_FC2 = 0x02
MOE_STAGE_DGRAD2 = 0x04
MOE_STAGE_WGRAD2 = 0x08
MOE_STAGE_DGRAD1 = 0x10
MOE_STAGE_WGRAD1 = 0x20
MOE_STAGES_FWD = MOE_STAGE_FC1 | MOE_STAGE_FC2
MOE_STAGES_BWD = MOE_STAGE_DGRAD2 | MOE_STAGE_WGRAD2 | MOE_STAGE_DGRAD1 | MOE_STAGE_WGRAD1
MOE_GATHER_ROWS = 0x100
MOE_ERRBIT_NONFINITE_LOGIT = 0x1
MOE_QUANT_ROWWISE = 0x1
MOE_QUANT_COLWISE = 0x2
MOE_ROUTE_STATIC_SCRATCH_BYTES = 8 << 20
MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1
MOE_MAX_TOPK = 64
MOE_MAX_GROUPS = 64
MOE_X_BF16 = 0
MOE_X_MXFP8 = 1
MOE_X_MXFP4 = 2
MOE_MAX_NORM_WIDTH = 16384
MOE_GATE_LINEAR = 0
MOE_GATE_SIGMOID = 1

# (name, restype, argtypes) of every exported symbol
_P = C.c_void_p
_I = C.c_int
_I64 = C.c_int64
_SZ = C.c_size_t
SIGNATURES = {
    "moe_status_str": (C.c_char_p, [_I]),
    "moe_capacity_rows": (_I64, [_I, _I, _I]),
    "moe_route_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_mlp_bwd_workspace_bytes": (_SZ, [_I, _I64]),
    "moe_route_counts": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "moe_route_counts_noalloc": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I64, _P, _P]),
    "moe_route_bwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_permute": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P]),
    "moe_combine": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_grouped_mlp_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I64, _I, C.c_uint, _P, _P, _P,
                                 _P, _P]),
    "moe_grouped_mlp_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I64, _I,
                                 C.c_uint, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "moe_quant_mxfp8": (_I, [_P, _I, _I64, _I, _I, _P, _P, _P, _P, _P]),
    "moe_permute_quant_mxfp8": (_I, [_P, _P, _I, _I, _I, _I, _I64, _I, _P, _P, _P, _P, _P]),
    "moe_linear_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_linear_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_act_bwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_linear_dgrad": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_linear_wgrad": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_dequant_mxfp8": (_I, [_P, _P, _I64, _I, _P, _P]),
    "moe_balance_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_balance_loss": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, C.c_float, C.c_float, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_balance_loss_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, C.c_float, C.c_float, _P, _I, _P, _P, _P]),
    "moe_route_scores_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_route_scores": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "moe_route_scores_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_quant_mxfp4": (_I, [_P, _I, _I64, _I, _I, _P, _P, _P, _P, _P]),
    "moe_dequant_mxfp4": (_I, [_P, _P, _I64, _I, _P, _P]),
    "moe_grouped_linear_mxfp4_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_grouped_linear_mxfp4": (_I, [_P, _P, _I, _P, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _P, _P, _SZ, _P]),
    "moe_norm_workspace_bytes": (_SZ, [_I, _I]),
    "moe_norm_fwd": (_I, [_P, _P, _P, _I, _I, C.c_float, _P, _P, _P, _P]),
    "moe_norm_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_post_norm_fwd": (_I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, C.c_float, C.c_float, _I, _I, _P, _P, _P, _P]),
    "moe_post_norm_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, C.c_float, _I, _I, _P, _P, _P, _P, _SZ, _P]),
}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {_lib().moe_status_str(status).decode()} ({status})")
        self.status = status


MX_FWD_FIELDS = ("a_q", "a_s", "at_q", "at_s", "w2t_q", "w2t_s", "x_q", "x_s", "w1t_q", "w1t_s",
                 "y_q", "y_s", "yt_q", "yt_s")
MX_BWD_FIELDS = ("dh_q", "dh_s", "dht_q", "dht_s", "awt_q", "awt_s", "dyt_q", "dyt_s", "xt_q", "xt_s",
                 "w1_q", "w1_s", "dy_q", "dy_s", "w2_q", "w2_s", "dx_q", "dx_s",
                 "dxt_q", "dxt_s")


class moe_mx_fwd(C.Structure):
    _fields_ = [(name, _P) for name in MX_FWD_FIELDS]


class moe_mx_bwd(C.Structure):
    _fields_ = [(name, _P) for name in MX_BWD_FIELDS]


class moe_routing(C.Structure):
    _fields_ = [("score", _I), ("groups", _I), ("topk_groups", _I), ("group_top", _I), ("renorm", _I), ("scale", C.c_float)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run ragged_grouped_gemm_device_amd.build")
        lib = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def load():
    """Load libmoe.so (raises if it is missing) and return the CDLL."""
    return _lib()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device=0):
    # the current stream's handle without building a torch.cuda.Stream (0.1 instead of 2.7 us)
    if device < 0:   # operands that agree with each other, but are none of a kernel's
        raise ValueError("the operands are not on a GPU")
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _check(fn: str, rc: int):
    if rc != MOE_OK:
        raise MoEError(fn, rc)


# ------------------------------------------------------------------ host-only
def moe_status_str(status: int) -> str:
    return _lib().moe_status_str(status).decode()


def moe_capacity_rows(T: int, k: int, E: int) -> int:
    return int(_lib().moe_capacity_rows(T, k, E))


def moe_route_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(_lib().moe_route_workspace_bytes(T, k, E))


def moe_mlp_bwd_workspace_bytes(n: int, M_cap: int) -> int:
    return int(_lib().moe_mlp_bwd_workspace_bytes(n, M_cap))


# ------------------------------------------------------------------ device calls
def moe_route_counts(logits, k, topk_idx, topk_w, counts, offsets, row_of, src_of, M_cap,
                     err_word, workspace, renorm=False):
    T, E = logits.shape
    rc = _lib().moe_route_counts(_ptr(logits), T, E, k, int(bool(renorm)), _ptr(topk_idx),
                                 _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(row_of),
                                 _ptr(src_of), M_cap, _ptr(err_word), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream())
    _check("moe_route_counts", rc)


def moe_route_counts_noalloc(logits, k, topk_idx, topk_w, counts, offsets, row_of, src_of, M_cap,
                             err_word, renorm=False):
    """moe_route_counts on the library's static scratch (no workspace argument)."""
    T, E = logits.shape
    rc = _lib().moe_route_counts_noalloc(_ptr(logits), T, E, k, int(bool(renorm)), _ptr(topk_idx),
                                         _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(row_of),
                                         _ptr(src_of), M_cap, _ptr(err_word), _stream())
    _check("moe_route_counts_noalloc", rc)


def moe_route_bwd(logits, topk_idx, ds, dlogits, renorm=False):
    T, E = logits.shape
    k = topk_idx.shape[1]
    rc = _lib().moe_route_bwd(_ptr(logits), _ptr(topk_idx), _ptr(ds), T, E, k, int(renorm),
                              _ptr(dlogits), _stream())
    _check("moe_route_bwd", rc)


def moe_permute(x, row_of, src_of, offsets, k, E, x_perm):
    T, d = x.shape
    rc = _lib().moe_permute(_ptr(x), _ptr(row_of), _ptr(src_of), _ptr(offsets), T, k, E, d,
                            x_perm.shape[0], _ptr(x_perm), _stream())
    _check("moe_permute", rc)


def moe_combine(y, row_of, w, k, out):
    T, d = out.shape
    rc = _lib().moe_combine(_ptr(y), _ptr(row_of), _ptr(w), T, k, d, _ptr(out), _stream())
    _check("moe_combine", rc)


def _fits(t, rows, cols, name):
    """The C ABI takes bare pointers: a tensor given for an operand of `cols` columns must be a
    dense [>= rows, cols] matrix (or [E, rows, cols] when rows is a tuple), else the kernels
    would address past it."""
    if t is None:
        return
    want = tuple(rows) + (cols,) if isinstance(rows, tuple) else None
    ok = t.is_contiguous() and (tuple(t.shape) == want if want else
                                t.dim() == 2 and t.shape[1] == cols and t.shape[0] >= rows)
    if not ok:
        raise ValueError(f"{name}: shape {tuple(t.shape)} does not fit "
                         f"{want if want else f'[>= {rows}, {cols}]'} (dense)")


def moe_grouped_mlp_fwd(x_perm, w1, w2, offsets, h, a, y, stages=MOE_STAGES_FWD, mx=None,
                        act=MOE_ACT_SWIGLU, src_of=None, k=0):
    """With MOE_GATHER_ROWS in stages, x_perm is the un-permuted x [T, d] and src_of, k are
    required."""
    E, d, n1 = w1.shape
    n = n1 if act == MOE_ACT_SRELU else n1 // 2
    M_cap = (a if a is not None else mx["a_q"]).shape[0]  # a may be None with mx
    T = x_perm.shape[0] if (stages & MOE_GATHER_ROWS) else 0
    if x_perm is not None:
        _fits(x_perm, T if (stages & MOE_GATHER_ROWS) else M_cap, d, "x_perm")
    _fits(w2, (E, n), d, "w2")
    _fits(h, M_cap, n1, "h")
    _fits(a, M_cap, n, "a")
    _fits(y, M_cap, d, "y")
    mxp = None
    if mx is not None:
        mxs = moe_mx_fwd(*[_ptr(mx.get(key)) for key in MX_FWD_FIELDS])
        mxp = C.byref(mxs)
    rc = _lib().moe_grouped_mlp_fwd(_ptr(x_perm), _ptr(w1), _ptr(w2), _ptr(offsets), _ptr(src_of), T,
                                    k, E, d, n, M_cap, act, stages, _ptr(h), _ptr(a), _ptr(y),
                                    mxp, _stream())
    _check("moe_grouped_mlp_fwd", rc)


def moe_grouped_mlp_bwd(x_perm, w1, w2, h, dy_u, topk_w, src_of, row_of, offsets, dh, a_w, ds,
                        dx_perm, dw1, dw2, workspace, stages=MOE_STAGES_BWD, act=MOE_ACT_SWIGLU,
                        mx=None, shape=None):
    """mx: dict of the moe_mx_bwd fields (missing ones pass NULL). shape = (E, d, n) when w1
    is not given (an MX call that reads only the quantized copies)."""
    if w1 is not None:
        E, d, n1 = w1.shape
        n = n1 if act == MOE_ACT_SRELU else n1 // 2
    else:
        E, d, n = shape
    mxp = None
    if mx is not None:
        mxp = C.byref(moe_mx_bwd(*[_ptr(mx.get(key)) for key in MX_BWD_FIELDS]))
    T, k = topk_w.shape
    M_cap = src_of.shape[0]
    n1 = n if act == MOE_ACT_SRELU else 2 * n
    rows_in = T if (stages & MOE_GATHER_ROWS) else M_cap
    _fits(x_perm, rows_in, d, "x_perm")
    _fits(dy_u, rows_in, d, "dy_u")
    _fits(w2, (E, n), d, "w2")
    _fits(h, M_cap, n1, "h")
    _fits(dh, M_cap, n1, "dh")
    _fits(a_w, M_cap, n, "a_w")
    _fits(dx_perm, M_cap, d, "dx_perm")
    _fits(dw1, (E, d), n1, "dw1")
    _fits(dw2, (E, n), d, "dw2")
    rc = _lib().moe_grouped_mlp_bwd(_ptr(x_perm), _ptr(w1), _ptr(w2), _ptr(h), _ptr(dy_u),
                                    _ptr(topk_w), _ptr(src_of), _ptr(row_of), _ptr(offsets), T, k,
                                    E, d, n, M_cap, act, stages, _ptr(dh), _ptr(a_w), _ptr(ds),
                                    _ptr(dx_perm), _ptr(dw1), _ptr(dw2), _ptr(workspace),
                                    0 if workspace is None else workspace.numel() * workspace.element_size(),
                                    mxp, _stream())
    _check("moe_grouped_mlp_bwd", rc)


def moe_quant_mxfp8(src, mode, q_row=None, s_row=None, q_col=None, s_col=None):
    if src.dim() == 2:
        batch, (R, Cc) = 1, src.shape
    else:
        batch, R, Cc = src.shape
    rc = _lib().moe_quant_mxfp8(_ptr(src), batch, R, Cc, mode, _ptr(q_row), _ptr(s_row),
                                _ptr(q_col), _ptr(s_col), _stream())
    _check("moe_quant_mxfp8", rc)


def moe_permute_quant_mxfp8(x, src_of, k, E, mode, q_row=None, s_row=None, q_col=None, s_col=None):
    T, d = x.shape
    rc = _lib().moe_permute_quant_mxfp8(_ptr(x), _ptr(src_of), T, k, E, d, src_of.shape[0], mode,
                                        _ptr(q_row), _ptr(s_row), _ptr(q_col), _ptr(s_col), _stream())
    _check("moe_permute_quant_mxfp8", rc)


# ------------------------------------------------------------------ dense half of the layer
_GATED = (MOE_ACT_SWIGLU, MOE_ACT_GEGLU)
_BF, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _operand(t, shape, dtype, name, device, other=None):
    """A tensor handed over by address must be exactly this dense matrix, on the device whose
    stream the call goes to (`other`: a second type that will do). A decode step makes several of
    these calls, so the test is one line."""
    if t is not None and not (t.shape == shape and (t.dtype is dtype or t.dtype is other) and t.is_contiguous()
                              and t.get_device() == device):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not dense'}; expected a dense {dtype} {tuple(shape)} "
                         f"{'on the host' if device < 0 else f'on cuda:{device}'}")


def _device(t):
    """The index of the call's device: that of its first operand, which has to be the current one
    (the kernels go to the current device's stream)."""
    dev = t.get_device()
    if dev >= 0 and dev != torch._C._cuda_getDevice():
        raise ValueError(f"operands are on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _sizes(T, *others):
    """Refuses a row count, and other sizes, that the C ABI's 32 bits would not hold."""
    if T > MOE_MAX_ROWS:
        raise ValueError(f"{T} rows; at most {MOE_MAX_ROWS}")
    if max(others) > 0x7fffffff:
        raise ValueError(f"a size of {max(others)}, past 32 bits")


def _space(ws, device):
    """(address, bytes) of a workspace tensor."""
    if ws is None:
        return None, 0
    if not ws.is_contiguous() or ws.get_device() != device:
        raise ValueError(f"workspace: needs a dense tensor on the operands' device, got {ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def moe_linear_workspace_bytes(T: int, K: int, N: int, passes: int = MOE_LINEAR_FWD | MOE_LINEAR_BWD) -> int:
    return int(_lib().moe_linear_workspace_bytes(T, K, N, passes))


def moe_linear_fwd(x, w, y, act=MOE_ACT_NONE, bias=None, residual=None, z=None, z_q=None, z_s=None,
                   workspace=None):
    """y = f(x w + bias) + residual; y is bf16 or fp32. z, or z_q and z_s, keep the pre-activation
    for the backward pass (as bf16, as an 8-bit checkpoint)."""
    dev = _device(x)
    (T, K), N = x.shape, w.shape[1]
    _sizes(T, K, N)
    out = (T, N // 2 if act in _GATED else N)
    _operand(x, (T, K), _BF, "x", dev)
    _operand(w, (K, N), _BF, "w", dev)
    _operand(y, out, _BF, "y", dev, _F32)
    _operand(bias, (N,), _BF, "bias", dev)
    _operand(residual, out, _BF, "residual", dev)
    _operand(z, (T, N), _BF, "z", dev)
    _operand(z_q, (T, N), _U8, "z_q", dev)
    _operand(z_s, (T, N // MOE_MX_BLOCK), _U8, "z_s", dev)
    ws, nws = _space(workspace, dev)
    rc = _lib().moe_linear_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(residual), T, K, N, act,
                               int(y is not None and y.dtype is _F32),
                               _ptr(y), _ptr(z), _ptr(z_q), _ptr(z_s), ws, nws, _stream(dev))
    _check("moe_linear_fwd", rc)


def moe_act_bwd(dy, dz, act=MOE_ACT_NONE, z=None, z_q=None, z_s=None, a=None, dbias=None, workspace=None):
    """dz = dy f'(z) with z as bf16 or from its 8-bit checkpoint; optionally a = f(z) and dbias =
    column sums of dz. dz (and dy, when only a is wanted) may be None."""
    ref = next((t for t in (z, z_q, dy) if t is not None), None)
    if ref is None:
        raise ValueError("neither dy nor z is given")
    dev = _device(ref)
    T, N = ref.shape
    _sizes(T, N)
    out = (T, N // 2 if act in _GATED else N)
    _operand(dy, out, _BF, "dy", dev)
    _operand(z, (T, N), _BF, "z", dev)
    _operand(z_q, (T, N), _U8, "z_q", dev)
    _operand(z_s, (T, N // MOE_MX_BLOCK), _U8, "z_s", dev)
    _operand(dz, (T, N), _BF, "dz", dev)
    _operand(a, out, _BF, "a", dev)
    _operand(dbias, (N,), _F32, "dbias", dev)
    ws, nws = _space(workspace, dev)
    rc = _lib().moe_act_bwd(_ptr(dy), _ptr(z), _ptr(z_q), _ptr(z_s), T, N, act, _ptr(dz), _ptr(a), _ptr(dbias),
                            ws, nws, _stream(dev))
    _check("moe_act_bwd", rc)


def moe_linear_dgrad(dz, w, dx, residual=None, workspace=None):
    """dx = dz w^T + residual (residual may be dx itself)."""
    dev = _device(dz)
    T, (K, N) = dz.shape[0], w.shape
    _sizes(T, K, N)
    _operand(dz, (T, N), _BF, "dz", dev)
    _operand(w, (K, N), _BF, "w", dev)
    _operand(dx, (T, K), _BF, "dx", dev)
    _operand(residual, (T, K), _BF, "residual", dev)
    ws, nws = _space(workspace, dev)
    _check("moe_linear_dgrad", _lib().moe_linear_dgrad(_ptr(dz), _ptr(w), _ptr(residual), T, K, N, _ptr(dx), ws,
                                                       nws, _stream(dev)))


def moe_linear_wgrad(x, dz, dw, x_q=None, x_s=None, accumulate=False, workspace=None):
    """dw = x^T dz (added to an fp32 dw with accumulate); x as bf16, or None with its 8-bit
    checkpoint x_q, x_s."""
    dev = _device(dz)
    (T, N), K = dz.shape, dw.shape[0]
    _sizes(T, K, N)
    _operand(x, (T, K), _BF, "x", dev)
    _operand(x_q, (T, K), _U8, "x_q", dev)
    _operand(x_s, (T, K // MOE_MX_BLOCK), _U8, "x_s", dev)
    _operand(dz, (T, N), _BF, "dz", dev)
    _operand(dw, (K, N), _BF, "dw", dev, _F32)
    ws, nws = _space(workspace, dev)
    _check("moe_linear_wgrad", _lib().moe_linear_wgrad(_ptr(x), _ptr(x_q), _ptr(x_s), _ptr(dz), T, K, N,
                                                       int(dw.dtype == _F32), int(bool(accumulate)), _ptr(dw), ws,
                                                       nws, _stream(dev)))


def moe_dequant_mxfp8(q, s, out):
    """bf16 values of row-wise MXFP8 codes (restores an 8-bit checkpoint)."""
    dev = _device(q)
    R, Cc = q.shape
    _sizes(0, Cc)   # R is 64-bit
    _operand(q, (R, Cc), _U8, "q", dev)
    _operand(s, (R, Cc // MOE_MX_BLOCK), _U8, "s", dev)
    _operand(out, (R, Cc), _BF, "out", dev)
    _check("moe_dequant_mxfp8", _lib().moe_dequant_mxfp8(_ptr(q), _ptr(s), R, Cc, _ptr(out), _stream(dev)))


def moe_balance_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return int(_lib().moe_balance_workspace_bytes(T, E, S))


def _sequences(seq_offsets, S, dev):
    _operand(seq_offsets, (S + 1,), _I32, "seq_offsets", dev)


def moe_balance_loss(logits, topk_idx, loss, counts, prob, tokens, workspace, balance_coef, z_coef, valid=None,
                     seq_offsets=None):
    """Router losses [total, balance, z] with the per-sequence expert counts [S, E], mean
    probabilities [S, E] and live tokens [S + 2] that the backward reads."""
    dev = _device(logits)
    (T, E), k, S = logits.shape, topk_idx.shape[1], counts.shape[0]
    _sizes(T, E, k, S)
    _operand(logits, (T, E), _F32, "logits", dev)
    _operand(topk_idx, (T, k), _I32, "topk_idx", dev)
    _operand(valid, (T,), _U8, "valid", dev, torch.bool)
    _sequences(seq_offsets, S, dev)
    _operand(loss, (3,), _F32, "loss", dev)
    _operand(counts, (S, E), _I32, "counts", dev)
    _operand(prob, (S, E), _F32, "prob", dev)
    _operand(tokens, (S + 2,), _I32, "tokens", dev)
    ws, nws = _space(workspace, dev)
    rc = _lib().moe_balance_loss(_ptr(logits), _ptr(topk_idx), _ptr(valid), _ptr(seq_offsets), T, E, k, S,
                                 balance_coef, z_coef, _ptr(loss), _ptr(counts), _ptr(prob), _ptr(tokens), ws, nws,
                                 _stream(dev))
    _check("moe_balance_loss", rc)


def moe_balance_loss_bwd(logits, counts, tokens, dlogits, k, balance_coef, z_coef, valid=None, seq_offsets=None,
                         grad=None, accumulate=False, dlogits_bf16=None):
    """Gradient of the total router loss w.r.t. the logits, written to (or, with accumulate, added
    to) dlogits; grad: the loss's upstream gradient (one fp32 value on the device)."""
    dev = _device(logits)
    (T, E), S = logits.shape, counts.shape[0]
    _sizes(T, E, k, S)
    _operand(logits, (T, E), _F32, "logits", dev)
    _operand(counts, (S, E), _I32, "counts", dev)
    _operand(tokens, (S + 2,), _I32, "tokens", dev)
    _operand(valid, (T,), _U8, "valid", dev, torch.bool)
    _sequences(seq_offsets, S, dev)
    _operand(dlogits, (T, E), _F32, "dlogits", dev)
    _operand(dlogits_bf16, (T, E), _BF, "dlogits_bf16", dev)
    if grad is not None:
        _operand(grad.reshape(1), (1,), _F32, "grad", dev)
    rc = _lib().moe_balance_loss_bwd(_ptr(logits), _ptr(counts), _ptr(tokens), _ptr(valid), _ptr(seq_offsets), T, E,
                                     k, S, balance_coef, z_coef, _ptr(grad), int(bool(accumulate)), _ptr(dlogits),
                                     _ptr(dlogits_bf16), _stream(dev))
    _check("moe_balance_loss_bwd", rc)


# ------------------------------------------------------------------ around the block
class Routing:
    """How tokens choose experts (moe_route_scores): scores (MOE_SCORE_*), a bias [E] fp32 that takes
    part in the choice alone (kept by reference; -inf takes an expert out of service), groups of
    neighbouring experts of which a token keeps topk_groups (a group is worth its best choice value, or
    with group_top = 2 the sum of its two best), and weights, renormalised over the chosen and scaled."""

    def __init__(self, score=MOE_SCORE_SIGMOID, bias=None, groups=1, topk_groups=1, group_top=2, renorm=True,
                 scale=1.0):
        self.bias = bias
        self.how = moe_routing(score, groups, topk_groups, group_top, int(bool(renorm)), scale)
        self.ref = C.byref(self.how)


def moe_route_scores_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(_lib().moe_route_scores_workspace_bytes(T, k, E))


def moe_route_scores(logits, k, topk_idx, topk_w, counts, offsets, row_of, src_of, err_word, workspace, routing):
    """moe_route_counts with the scores, bias, groups and weights of a Routing."""
    dev = _device(logits)
    T, E = logits.shape
    _sizes(T, E, k)
    _operand(logits, (T, E), _F32, "logits", dev)
    _operand(routing.bias, (E,), _F32, "bias", dev)
    _operand(topk_idx, (T, k), _I32, "topk_idx", dev)
    _operand(topk_w, (T, k), _F32, "topk_w", dev)
    _operand(counts, (E,), _I32, "counts", dev)
    _operand(offsets, (E + 1,), _I32, "offsets", dev)
    _operand(row_of, (T * k,), _I32, "row_of", dev)
    _operand(src_of, (src_of.numel(),), _I32, "src_of", dev)
    _operand(err_word, (1,), _I32, "err_word", dev)
    ws, nws = _space(workspace, dev)
    _check("moe_route_scores", _lib().moe_route_scores(
        _ptr(logits), _ptr(routing.bias), routing.ref, T, E, k, _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
        _ptr(offsets), _ptr(row_of), _ptr(src_of), src_of.numel(), _ptr(err_word), ws, nws, _stream(dev)))


def moe_route_scores_bwd(logits, topk_idx, ds, dlogits, routing):
    """dlogits [T, E] from ds = dL/dtopk_w, for the experts that moe_route_scores chose."""
    dev = _device(logits)
    (T, E), k = logits.shape, topk_idx.shape[1]
    _sizes(T, E, k)
    _operand(logits, (T, E), _F32, "logits", dev)
    _operand(routing.bias, (E,), _F32, "bias", dev)
    _operand(topk_idx, (T, k), _I32, "topk_idx", dev)
    _operand(ds, (T, k), _F32, "ds", dev)
    _operand(dlogits, (T, E), _F32, "dlogits", dev)
    _check("moe_route_scores_bwd", _lib().moe_route_scores_bwd(
        _ptr(logits), _ptr(routing.bias), routing.ref, _ptr(topk_idx), _ptr(ds), T, E, k, _ptr(dlogits), _stream(dev)))


def moe_quant_mxfp4(src, mode, q_row=None, s_row=None, q_col=None, s_col=None):
    """MXFP4 codes (two a byte) and scales of src [R, C] or [batch, R, C]: row-wise [.., R, C / 2] and
    [.., R, C / 32], column-wise and transposed [.., C, R / 2] and [.., C, R / 32]."""
    dev = _device(src)
    lead, (R, Cc) = tuple(src.shape[:-2]), src.shape[-2:]
    batch = lead[0] if lead else 1
    _sizes(0, Cc, batch)
    if src.dim() not in (2, 3):
        raise ValueError(f"src: {src.dim()} dimensions; 2 or 3 expected")
    _operand(src, src.shape, _BF, "src", dev)
    _operand(q_row, lead + (R, Cc // 2), _U8, "q_row", dev)
    _operand(s_row, lead + (R, Cc // MOE_MX_BLOCK), _U8, "s_row", dev)
    _operand(q_col, lead + (Cc, R // 2), _U8, "q_col", dev)
    _operand(s_col, lead + (Cc, R // MOE_MX_BLOCK), _U8, "s_col", dev)
    _check("moe_quant_mxfp4", _lib().moe_quant_mxfp4(_ptr(src), batch, R, Cc, mode, _ptr(q_row), _ptr(s_row),
                                                     _ptr(q_col), _ptr(s_col), _stream(dev)))


def moe_dequant_mxfp4(q, s, out):
    """bf16 values [R, C] of row-wise MXFP4 codes [R, C / 2] and scales [R, C / 32]."""
    dev = _device(out)
    R, Cc = out.shape
    _sizes(0, Cc)
    _operand(q, (R, Cc // 2), _U8, "q", dev)
    _operand(s, (R, Cc // MOE_MX_BLOCK), _U8, "s", dev)
    _operand(out, (R, Cc), _BF, "out", dev)
    _check("moe_dequant_mxfp4", _lib().moe_dequant_mxfp4(_ptr(q), _ptr(s), R, Cc, _ptr(out), _stream(dev)))


def moe_grouped_linear_mxfp4_workspace_bytes(T: int, k: int, E: int, K: int, N: int) -> int:
    return int(_lib().moe_grouped_linear_mxfp4_workspace_bytes(T, k, E, K, N))


def moe_grouped_linear_mxfp4(x, w_q, w_s, offsets, counts, y, T, k, act=MOE_ACT_NONE, x_s=None, src_of=None,
                             workspace=None):
    """y = f(x W_e) for every expert's rows, W_e as MXFP4 [E, N, K / 2] with scales [E, N, K / 32]. x: the
    experts' rows [M_cap, ..], or with src_of the tokens [T, ..]; bf16, or codes with their scales x_s
    (MXFP8 [.., K], MXFP4 [.., K / 2]). y [M_cap, N], or [M_cap, N / 2] for a gated activation; rows past an
    expert's count are left as they are."""
    dev = _device(x)
    E, N, K = w_q.shape[0], w_q.shape[1], 2 * w_q.shape[2]
    _sizes(T, E, K, N, k)
    M_cap = y.shape[0]
    rows = M_cap if src_of is None else T
    fmt = MOE_X_BF16 if x_s is None else MOE_X_MXFP8 if x.shape[-1] == K else MOE_X_MXFP4
    _operand(x, (rows, K // 2 if fmt == MOE_X_MXFP4 else K), _BF if fmt == MOE_X_BF16 else _U8, "x", dev)
    _operand(x_s, (rows, K // MOE_MX_BLOCK), _U8, "x_s", dev)
    _operand(w_q, (E, N, K // 2), _U8, "w_q", dev)
    _operand(w_s, (E, N, K // MOE_MX_BLOCK), _U8, "w_s", dev)
    _operand(offsets, (E + 1,), _I32, "offsets", dev)
    _operand(counts, (E,), _I32, "counts", dev)
    _operand(src_of, (M_cap,), _I32, "src_of", dev)
    _operand(y, (M_cap, N // 2 if act in _GATED else N), _BF, "y", dev)
    ws, nws = _space(workspace, dev)
    _check("moe_grouped_linear_mxfp4", _lib().moe_grouped_linear_mxfp4(
        _ptr(x), _ptr(x_s), fmt, _ptr(src_of), T, k, _ptr(w_q), _ptr(w_s), _ptr(offsets), _ptr(counts), E, K, N, M_cap,
        act, _ptr(y), ws, nws, _stream(dev)))


def moe_norm_workspace_bytes(T: int, d: int) -> int:
    return int(_lib().moe_norm_workspace_bytes(T, d))


def moe_norm_fwd(x, w, y, rstd=None, eps=1e-6, residual=None, total=None):
    """total = x + residual (bf16), y = total rstd w; without a residual, x itself is normalised."""
    dev = _device(x)
    T, d = x.shape
    _sizes(T, d)
    _operand(x, (T, d), _BF, "x", dev)
    _operand(residual, (T, d), _BF, "residual", dev)
    _operand(w, (d,), _BF, "w", dev)
    _operand(total, (T, d), _BF, "total", dev)
    _operand(y, (T, d), _BF, "y", dev)
    _operand(rstd, (T,), _F32, "rstd", dev)
    _check("moe_norm_fwd", _lib().moe_norm_fwd(_ptr(x), _ptr(residual), _ptr(w), T, d, eps, _ptr(total), _ptr(y),
                                               _ptr(rstd), _stream(dev)))


def moe_norm_bwd(dy, x, w, rstd, dx, dw=None, workspace=None, dres=None):
    """dx (+ dres, the residual stream's gradient) and dw of a norm of x."""
    dev = _device(dy)
    T, d = dy.shape
    _sizes(T, d)
    for t, name in ((dy, "dy"), (x, "x"), (dres, "dres"), (dx, "dx")):
        _operand(t, (T, d), _BF, name, dev)
    _operand(w, (d,), _BF, "w", dev)
    _operand(rstd, (T,), _F32, "rstd", dev)
    _operand(dw, (d,), _F32, "dw", dev)
    ws, nws = _space(workspace, dev)
    _check("moe_norm_bwd", _lib().moe_norm_bwd(_ptr(dy), _ptr(x), _ptr(w), _ptr(rstd), _ptr(dres), T, d, _ptr(dx),
                                               _ptr(dw), ws, nws, _stream(dev)))


def _gate(gate, T, d, dev):
    """Columns of a post norm's gate: 0 (none), 1 (one a token) or d."""
    if gate is None:
        return 0
    cols = gate.shape[1] if gate.dim() == 2 else -1
    if cols not in (1, d):
        raise ValueError(f"gate: {tuple(gate.shape)}; expected {(T, 1)} or {(T, d)}")
    _operand(gate, (T, cols), _BF, "gate", dev)
    return cols


def moe_post_norm_fwd(y, x, w, out, rstd=None, eps=1e-6, gate=None, gate_act=MOE_GATE_LINEAR, scale=1.0, row_of=None,
                      topk_w=None, total=None):
    """out = x + scale f(gate) (norm(y) w). With row_of [T * k], y holds the experts' rows and their sum
    weighted by topk_w [T, k] is normalised (and stored in total)."""
    dev = _device(x)
    T, d = x.shape
    _sizes(T, d)
    k = 0
    if row_of is None:
        _operand(y, (T, d), _BF, "y", dev)
    else:
        k = row_of.numel() // max(T, 1)
        _operand(row_of, (T * k,), _I32, "row_of", dev)
        _operand(y, (y.shape[0], d), _BF, "y", dev)
        _operand(topk_w, (T, k), _F32, "topk_w", dev)
    for t, name in ((x, "x"), (total, "total"), (out, "out")):
        _operand(t, (T, d), _BF, name, dev)
    _operand(w, (d,), _BF, "w", dev)
    _operand(rstd, (T,), _F32, "rstd", dev)
    cols = _gate(gate, T, d, dev)
    _check("moe_post_norm_fwd", _lib().moe_post_norm_fwd(
        _ptr(y), _ptr(row_of), _ptr(topk_w), k, _ptr(x), _ptr(w), _ptr(gate), cols, gate_act, scale, eps, T, d,
        _ptr(total), _ptr(out), _ptr(rstd), _stream(dev)))


def moe_post_norm_bwd(dout, y, w, rstd, dy, dw=None, workspace=None, gate=None, dgate=None, gate_act=MOE_GATE_LINEAR,
                      scale=1.0):
    """Gradients of the block's output y, the gate (bf16 [T, d], fp32 [T, 1]) and w; x's is dout."""
    dev = _device(dout)
    T, d = dout.shape
    _sizes(T, d)
    for t, name in ((dout, "dout"), (y, "y"), (dy, "dy")):
        _operand(t, (T, d), _BF, name, dev)
    _operand(w, (d,), _BF, "w", dev)
    _operand(rstd, (T,), _F32, "rstd", dev)
    _operand(dw, (d,), _F32, "dw", dev)
    cols = _gate(gate, T, d, dev)
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate: there is no gate")
        _operand(dgate, (T, cols), _F32 if cols == 1 else _BF, "dgate", dev)
    ws, nws = _space(workspace, dev)
    _check("moe_post_norm_bwd", _lib().moe_post_norm_bwd(
        _ptr(dout), _ptr(y), _ptr(w), _ptr(rstd), _ptr(gate), cols, gate_act, scale, T, d, _ptr(dy), _ptr(dgate),
        _ptr(dw), ws, nws, _stream(dev)))


# ------------------------------------------------------------------ buffers
class Buffers:
    """Device buffers of one forward + backward pass (plain torch allocations)."""

    def __init__(self, T: int, k: int, E: int, d: int, n: int, device="cuda", mx: bool = False,
                 gated: bool = True, ckpt8: bool = False, h=None):
        """ckpt8: keep the FC1 output H between forward and backward as an 8-bit checkpoint (33
        instead of 64 bytes for 32 values); H itself is then scratch, and layers run one after the
        other may share one: pass it as h."""
        dev = torch.device(device)
        bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
        self.T, self.k, self.E, self.d, self.n = T, k, E, d, n
        self.M_cap = M = moe_capacity_rows(T, k, E)
        self.topk_idx = torch.empty(T, k, dtype=i32, device=dev)
        self.topk_w = torch.empty(T, k, dtype=f32, device=dev)
        self.counts = torch.empty(E, dtype=i32, device=dev)
        self.offsets = torch.empty(E + 1, dtype=i32, device=dev)
        self.row_of = torch.empty(T * k, dtype=i32, device=dev)
        self.src_of = torch.empty(M, dtype=i32, device=dev)
        self.err = torch.zeros(1, dtype=i32, device=dev)
        self.route_ws = torch.empty(max(16, moe_route_workspace_bytes(T, k, E), moe_route_scores_workspace_bytes(T, k, E)),
                                    dtype=u8, device=dev)
        self.x_perm = torch.empty(M, d, dtype=bf, device=dev)
        n1 = 2 * n if gated else n   # FC1 width (non-gated sReLU: n)
        if h is not None and not (h.shape == (M, n1) and h.dtype is bf and h.is_contiguous()
                                  and h.device.type == dev.type and dev.index in (None, h.device.index)):
            raise ValueError(f"h: {h.dtype} {tuple(h.shape)} on {h.device}; expected a dense {bf} {(M, n1)} on {dev}")
        self.h = torch.empty(M, n1, dtype=bf, device=dev) if h is None else h
        self.ckpt8 = ckpt8
        if ckpt8:
            self.h_q = torch.empty(M, n1, dtype=u8, device=dev)
            self.h_s = torch.empty(M, n1 // MOE_MX_BLOCK, dtype=u8, device=dev)
        self.a = torch.empty(M, n, dtype=bf, device=dev)
        self.y = torch.empty(M, d, dtype=bf, device=dev)
        self.out = torch.empty(T, d, dtype=bf, device=dev)
        self.dy_u = torch.empty(M, d, dtype=bf, device=dev)
        self.dh = torch.empty(M, n1, dtype=bf, device=dev)
        self.a_w = torch.empty(M, n, dtype=bf, device=dev)
        self.ds = torch.empty(T, k, dtype=f32, device=dev)
        self.dx_perm = torch.empty(M, d, dtype=bf, device=dev)
        self.dx = torch.empty(T, d, dtype=bf, device=dev)
        self.dw1 = torch.empty(E, d, n1, dtype=f32, device=dev)
        self.dw2 = torch.empty(E, n, d, dtype=f32, device=dev)
        self.dlogits = torch.empty(T, E, dtype=f32, device=dev)
        self.bwd_ws = torch.empty(max(16, moe_mlp_bwd_workspace_bytes(n, M)), dtype=u8, device=dev)
        if mx:
            self.a_q = torch.empty(M, n, dtype=u8, device=dev)
            self.a_s = torch.empty(M, n // 32, dtype=u8, device=dev)
            self.at_q = torch.empty(n, M, dtype=u8, device=dev)
            self.at_s = torch.empty(n, M // 32, dtype=u8, device=dev)
            self.w2t_q = torch.empty(E, d, n, dtype=u8, device=dev)
            self.w2t_s = torch.empty(E, d, n // 32, dtype=u8, device=dev)
            self.dh_q = torch.empty(M, 2 * n, dtype=u8, device=dev)
            self.dh_s = torch.empty(M, 2 * n // 32, dtype=u8, device=dev)
            self.dht_q = torch.empty(2 * n, M, dtype=u8, device=dev)
            self.dht_s = torch.empty(2 * n, M // 32, dtype=u8, device=dev)
            self.awt_q = torch.empty(n, M, dtype=u8, device=dev)
            self.awt_s = torch.empty(n, M // 32, dtype=u8, device=dev)
            self.dyt_q = torch.empty(d, M, dtype=u8, device=dev)
            self.dyt_s = torch.empty(d, M // 32, dtype=u8, device=dev)
            self.xt_q = torch.empty(d, M, dtype=u8, device=dev)
            self.xt_s = torch.empty(d, M // 32, dtype=u8, device=dev)
            self.w1_q = torch.empty(E, d, 2 * n, dtype=u8, device=dev)
            self.w1_s = torch.empty(E, d, 2 * n // 32, dtype=u8, device=dev)
            self.x_q = torch.empty(M, d, dtype=u8, device=dev)
            self.x_s = torch.empty(M, d // 32, dtype=u8, device=dev)
            self.w1t_q = torch.empty(E, 2 * n, d, dtype=u8, device=dev)
            self.w1t_s = torch.empty(E, 2 * n, d // 32, dtype=u8, device=dev)
            self.dy_q = torch.empty(M, d, dtype=u8, device=dev)
            self.dy_s = torch.empty(M, d // 32, dtype=u8, device=dev)
            self.w2_q = torch.empty(E, n, d, dtype=u8, device=dev)
            self.w2_s = torch.empty(E, n, d // 32, dtype=u8, device=dev)
            # row-wise MXFP8 copies of the FC2 output and of the FC1 dgrad output
            # (GroupGemm + Quantize), written only when asked
            self.y_q = torch.empty(M, d, dtype=u8, device=dev)
            self.y_s = torch.empty(M, d // 32, dtype=u8, device=dev)
            self.dx_q = torch.empty(M, d, dtype=u8, device=dev)
            self.dx_s = torch.empty(M, d // 32, dtype=u8, device=dev)
            # and their column-wise copies, transposed
            self.yt_q = torch.empty(d, M, dtype=u8, device=dev)
            self.yt_s = torch.empty(d, M // 32, dtype=u8, device=dev)
            self.dxt_q = torch.empty(d, M, dtype=u8, device=dev)
            self.dxt_s = torch.empty(d, M // 32, dtype=u8, device=dev)
        self.xt_from_forward = False
        self.served = False   # the last forward kept nothing for a backward pass

    def quantize_weights(self, w1, w2):
        """MXFP8 weight copies: W1_e along 2n [E, d, 2n] (FC1 dgrad) and along d, transposed
        [E, 2n, d] (FC1); W2_e along d [E, n, d] (FC2 dgrad) and along n, transposed [E, d, n]
        (FC2)."""
        moe_quant_mxfp8(w1, MOE_QUANT_ROWWISE | MOE_QUANT_COLWISE, self.w1_q, self.w1_s, self.w1t_q,
                        self.w1t_s)
        moe_quant_mxfp8(w2, MOE_QUANT_ROWWISE | MOE_QUANT_COLWISE, self.w2_q, self.w2_s, self.w2t_q,
                        self.w2t_s)

    def mx_fwd(self, fc1=True, transposed_a=False, quant_y=False, transposed_y=False):
        """The moe_mx_fwd fields: FC1 on MXFP8 operands when fc1; the transposed copy of A
        only when asked (the training step's FC2 wgrad reads A' = w A, quantized by the FC2
        dgrad, not A); the row-wise MXFP8 copy of Y (FC2 epilogue) when quant_y, with its
        transposed column-wise copy when transposed_y."""
        keys = MX_FWD_FIELDS[:10] if fc1 else MX_FWD_FIELDS[:6]
        d = {key: getattr(self, key) for key in keys}
        if not transposed_a:
            d["at_q"] = d["at_s"] = None
        if quant_y:
            d["y_q"], d["y_s"] = self.y_q, self.y_s
            if transposed_y:
                d["yt_q"], d["yt_s"] = self.yt_q, self.yt_s
        return d

    def mx_bwd(self, dgrad2=True, quant_dx=False, transposed_dx=False):
        keys = MX_BWD_FIELDS[:16] if dgrad2 else MX_BWD_FIELDS[:12]
        d = {key: getattr(self, key) for key in keys}
        if quant_dx:
            d["dx_q"], d["dx_s"] = self.dx_q, self.dx_s
            if transposed_dx:
                d["dxt_q"], d["dxt_s"] = self.dxt_q, self.dxt_s
        return d


class SharedExpert:
    """The expert every token passes, beside the routed ones: out += f(x w1) w2, with w1 [d, 2n]
    (gated; interleaved like the routed experts' W1) or [d, n], w2 [n, d]. Between forward and
    backward it keeps z = x w1 as an 8-bit checkpoint (ckpt8) or as bf16; f(z) is recomputed. With
    x8 it keeps an 8-bit checkpoint of x too, and the backward needs no x. out and dx are rounded to
    bf16 with the routed part in them and once more with this expert's added; dw1 and dw2 are
    written, not added to."""

    def __init__(self, T: int, d: int, n: int, act: int = MOE_ACT_SWIGLU, ckpt8: bool = True, x8: bool = False,
                 device="cuda"):
        self.act, self.x8 = act, x8
        n1 = 2 * n if act in _GATED else n
        new = lambda *shape, t=_BF: torch.empty(*shape, dtype=t, device=device)  # noqa: E731
        self.z = None if ckpt8 else new(T, n1)
        self.z_q = new(T, n1, t=_U8) if ckpt8 else None
        self.z_s = new(T, n1 // MOE_MX_BLOCK, t=_U8) if ckpt8 else None
        self.x_q = new(T, d, t=_U8) if x8 else None
        self.x_s = new(T, d // MOE_MX_BLOCK, t=_U8) if x8 else None
        self.a, self.da, self.dz = new(T, n), new(T, n), new(T, n1)
        self.dw1, self.dw2 = new(d, n1, t=_F32), new(n, d, t=_F32)
        size = max(16, moe_linear_workspace_bytes(T, d, n1), moe_linear_workspace_bytes(T, n, d))
        self.ws = new(size, t=_U8)

    def forward(self, x, w1, w2, out):
        """out += f(x w1) w2."""
        moe_linear_fwd(x, w1, self.a, self.act, z=self.z, z_q=self.z_q, z_s=self.z_s, workspace=self.ws)
        if self.x8:
            moe_quant_mxfp8(x, MOE_QUANT_ROWWISE, self.x_q, self.x_s)
        moe_linear_fwd(self.a, w2, out, residual=out, workspace=self.ws)

    def backward(self, x, dout, w1, w2, dx):
        """dw1, dw2, and dx += the gradient through the shared expert."""
        moe_linear_dgrad(dout, w2, self.da, workspace=self.ws)
        moe_act_bwd(self.da, self.dz, self.act, z=self.z, z_q=self.z_q, z_s=self.z_s, a=self.a)
        moe_linear_wgrad(self.a, dout, self.dw2, workspace=self.ws)
        moe_linear_dgrad(self.dz, w1, dx, residual=dx, workspace=self.ws)
        moe_linear_wgrad(None if self.x8 else x, self.dz, self.dw1, x_q=self.x_q, x_s=self.x_s, workspace=self.ws)


class Router:
    """The router's projection logits = x wg (wg [d, E]) with the balance and z losses of the
    routing: loss [total, balance, z], counts, prob and tokens after forward; dwg after backward.
    Sequences and padding tokens: seq_offsets [S + 1] and valid [T], kept by reference (set them
    before a forward). The products take widths in steps of 8: with another E they work on copies
    with columns of zeros behind it."""

    def __init__(self, T: int, d: int, E: int, k: int, S: int = 1, balance_coef: float = 1e-2,
                 z_coef: float = 1e-3, device="cuda"):
        self.k, self.balance_coef, self.z_coef = k, balance_coef, z_coef
        new = lambda *shape, t=_F32: torch.empty(*shape, dtype=t, device=device)  # noqa: E731
        self.logits, self.dlogits16, self.dwg = new(T, E), new(T, E, t=_BF), new(d, E)
        self.loss, self.counts, self.prob = new(3), new(S, E, t=_I32), new(S, E)
        self.tokens = new(S + 2, t=_I32)
        self.valid = self.seq_offsets = None
        self.wide = None
        N = -(-E // 8) * 8
        if N != E:   # wg, logits, dlogits16 and dwg as the products take them
            self.wide = (new(d, N, t=_BF).zero_(), new(T, N), new(T, N, t=_BF).zero_(), new(d, N))
        self.ws = new(max(16, moe_linear_workspace_bytes(T, d, N)), t=_U8)
        self.loss_ws = new(moe_balance_workspace_bytes(T, E, S), t=_U8)

    def _weight(self, wg):
        if self.wide is None:
            return wg
        _operand(wg, self.dwg.shape, _BF, "wg", self.logits.get_device())
        self.wide[0][:, :wg.shape[1]].copy_(wg.detach())
        return self.wide[0]

    def project(self, x, wg):
        wg, out = self._weight(wg), self.logits if self.wide is None else self.wide[1]
        moe_linear_fwd(x, wg, out, workspace=self.ws)
        if out is not self.logits:
            self.logits.copy_(out[:, :self.logits.shape[1]])
        return self.logits

    def losses(self, topk_idx):
        if topk_idx.shape[1] != self.k:   # the backward's f_se divides by self.k
            raise ValueError(f"topk_idx: {topk_idx.shape[1]} experts a token; the router was made with k = {self.k}")
        moe_balance_loss(self.logits, topk_idx, self.loss, self.counts, self.prob, self.tokens, self.loss_ws,
                         self.balance_coef, self.z_coef, valid=self.valid, seq_offsets=self.seq_offsets)

    def backward(self, x, wg, dlogits, dx, grad=None):
        """dlogits += the losses' gradient (times grad, their upstream gradient); dwg; dx += the
        gradient through the projection. Both products run on bf16 matrix cores and take the fp32
        dlogits rounded to bf16, so dwg, though fp32, is off by up to 2^-8 of each term; dwg is
        written, not added to."""
        moe_balance_loss_bwd(self.logits, self.counts, self.tokens, dlogits, self.k, self.balance_coef, self.z_coef,
                             valid=self.valid, seq_offsets=self.seq_offsets, grad=grad, accumulate=True,
                             dlogits_bf16=self.dlogits16)
        wg, E = self._weight(wg), self.logits.shape[1]
        d16, dwg = (self.dlogits16, self.dwg) if self.wide is None else self.wide[2:]
        if d16 is not self.dlogits16:
            d16[:, :E].copy_(self.dlogits16)
        moe_linear_dgrad(d16, wg, dx, residual=dx, workspace=self.ws)
        moe_linear_wgrad(x, d16, dwg, workspace=self.ws)
        if dwg is not self.dwg:
            self.dwg.copy_(dwg[:, :E])


def _used_rows(T: int, k: int, E: int) -> int:
    """Rows of the experts' buffer that a routing of T tokens can reach: those of the experts hit, each up to its
    region's end. Few tokens hit few of many experts, and the capacity is for all."""
    return (T * k + (MOE_ALIGN - 1) * min(E, T * k)) // MOE_ALIGN * MOE_ALIGN


class Experts4:
    """The routed experts' weights as MXFP4, for serving: w1 [E, d, 2n] (gated; n wide otherwise) and w2
    [E, n, d] in 17 instead of 64 bytes for 32 values. x_form: how the products take their rows, as bf16, or
    quantized to MXFP8 or MXFP4 on the way (the tokens once, before they are gathered). It serves calls of T
    tokens, one at a time: the rows' codes and the workspace are its own. sized(T) gives one for another number of
    tokens, or another stream, on the same weights."""

    def __init__(self, T: int, k: int, E: int, d: int, n: int, act: int = MOE_ACT_SWIGLU, x_form: int = MOE_X_BF16,
                 device="cuda"):
        self.k, self.act, self.x_form = k, act, x_form
        n1 = 2 * n if act in _GATED else n
        new = lambda *shape: torch.empty(*shape, dtype=_U8, device=device)  # noqa: E731
        self.w1_q, self.w1_s = new(E, n1, d // 2), new(E, n1, d // MOE_MX_BLOCK)
        self.w2_q, self.w2_s = new(E, d, n // 2), new(E, d, n // MOE_MX_BLOCK)
        self._scratch(T)

    def _scratch(self, T):
        (E, n1, d), n = self.w1_s.shape, self.w2_q.shape[2] * 2
        d *= MOE_MX_BLOCK
        new = lambda *shape: torch.empty(*shape, dtype=_U8, device=self.w1_q.device)  # noqa: E731
        self.T = T
        M = moe_capacity_rows(T, self.k, E)
        self.x_q = self.x_s = self.a_q = self.a_s = None
        if self.x_form != MOE_X_BF16:
            per = 1 if self.x_form == MOE_X_MXFP8 else 2
            self.x_q, self.x_s = new(T, d // per), new(T, d // MOE_MX_BLOCK)
            self.a_q, self.a_s = new(M, n // per), new(M, n // MOE_MX_BLOCK)
            self.used = _used_rows(T, self.k, E)
        self.ws = new(max(16, moe_grouped_linear_mxfp4_workspace_bytes(T, self.k, E, d, n1),
                          moe_grouped_linear_mxfp4_workspace_bytes(T, self.k, E, n, d)))

    def sized(self, T: int):
        """An Experts4 for T tokens a call on these weights (the same tensors: load on either fills both), with
        codes and workspace of its own, so that both may run at once."""
        other = copy.copy(self)
        other._scratch(T)
        return other

    def load(self, w1, w2):
        """Quantizes bf16 weights, once."""
        moe_quant_mxfp4(w1, MOE_QUANT_COLWISE, q_col=self.w1_q, s_col=self.w1_s)
        moe_quant_mxfp4(w2, MOE_QUANT_COLWISE, q_col=self.w2_q, s_col=self.w2_s)

    def _rows(self, x, q, s, used=None):
        if self.x_form == MOE_X_BF16:
            return x, None
        quant = moe_quant_mxfp8 if self.x_form == MOE_X_MXFP8 else moe_quant_mxfp4
        quant(x[:used], MOE_QUANT_ROWWISE, q[:used], s[:used])
        return q, s

    def forward(self, x, offsets, counts, src_of, a, y):
        """a = f(x w1), y = a w2 over the rows that the routing made."""
        q, s = self._rows(x, self.x_q, self.x_s)
        moe_grouped_linear_mxfp4(q, self.w1_q, self.w1_s, offsets, counts, a, self.T, self.k, act=self.act, x_s=s,
                                 src_of=src_of, workspace=self.ws)
        # of rows between those that the routing made, the codes are of whatever the buffer holds, and not read
        q, s = self._rows(a, self.a_q, self.a_s, None if self.a_q is None else self.used)
        moe_grouped_linear_mxfp4(q, self.w2_q, self.w2_s, offsets, counts, y, self.T, self.k, x_s=s, workspace=self.ws)


class BlockNorms:
    """The norms of the residual block around the layer: out = x + scale f(gate) (norm(layer(norm(x) w_pre)) w_post).
    After a forward: out, and y, the layer's input; after a backward: dx, dw_pre, dw_post, and dgate (bf16 [T, d],
    or fp32 [T, 1] for one gate a token). gate_cols: 0 (no gate), 1 or d."""

    def __init__(self, T: int, d: int, gate_cols: int = 0, gate_act: int = MOE_GATE_LINEAR, scale: float = 1.0,
                 eps: float = 1e-6, device="cuda"):
        new = lambda *shape, t=_BF: torch.empty(*shape, dtype=t, device=device)  # noqa: E731
        self.gate_act, self.scale, self.eps = gate_act, scale, eps
        self.y, self.out, self.dy, self.dx = new(T, d), new(T, d), new(T, d), new(T, d)
        self.rstd_pre, self.rstd_post = new(T, t=_F32), new(T, t=_F32)
        self.dw_pre, self.dw_post = new(d, t=_F32), new(d, t=_F32)
        self.dgate = new(T, gate_cols, t=_F32 if gate_cols == 1 else _BF) if gate_cols else None
        self.ws = new(max(16, moe_norm_workspace_bytes(T, d)), t=_U8)

    def before(self, x, w):
        moe_norm_fwd(x, w, self.y, self.rstd_pre, self.eps)
        return self.y

    def after(self, x, w, gate, y, **rows):
        moe_post_norm_fwd(y, x, w, self.out, self.rstd_post, self.eps, gate=gate, gate_act=self.gate_act,
                          scale=self.scale, **rows)

    def back_after(self, dout, w, gate, y):
        if gate is not None and self.dgate is None:
            raise ValueError("gate: its gradient has no place, gate_cols was 0")
        moe_post_norm_bwd(dout, y, w, self.rstd_post, self.dy, self.dw_post, self.ws, gate=gate, dgate=self.dgate,
                          gate_act=self.gate_act, scale=self.scale)
        return self.dy

    def back_before(self, dy, dout, x, w):
        moe_norm_bwd(dy, x, w, self.rstd_pre, self.dx, self.dw_pre, self.ws, dres=dout)


def _check_losses(router, routing):
    if router is not None and routing is not None and routing.how.score == MOE_SCORE_SIGMOID and router[0].balance_coef:
        raise ValueError("the Router's balance loss is that of softmax probabilities: with sigmoid scores, balance_coef=0")


def forward(buf: Buffers, x, logits, w1, w2, renorm=False, fwd_stages=MOE_STAGES_FWD, store_h=True,
            act=MOE_ACT_SWIGLU, gather=False, mx=False, router=None, shared=None, routing=None, experts4=None,
            norms=None):
    """route -> permute -> FC1+GLU -> FC2 -> combine (all enqueued, no sync). With gather, FC1
    reads the rows of x through src_of and no permuted copy is made. With mx (buffers made with
    mx=True, quantize_weights done), X_perm is quantized row-wise (FC1 operand) and column-wise
    (FC1 wgrad operand) in one pass and both GEMMs run on MXFP8. With buffers made with ckpt8, H
    is kept as an 8-bit checkpoint. router = (Router, wg): the logits are x wg (logits is None),
    and the router losses follow the routing. shared = (SharedExpert, w1, w2): the shared expert's
    output is added to out. routing = a Routing: its scores, bias, groups and weights (renorm is then its
    own); a Router beside sigmoid scores needs balance_coef = 0, as its balance loss is a softmax's.
    experts4 = an Experts4 (serving): its 4-bit weights and activation in place of w1, w2 and act; it reads the
    rows of x through src_of, with gather or without, and nothing is kept for a backward pass, whatever store_h
    says; mx, and single stages, are refused. norms = (BlockNorms, w_pre, w_post, gate or None): x is the residual
    stream, the layer runs on its norm, buf.out holds the layer's output and the BlockNorms' out the block's."""
    if experts4 is not None:
        if mx or fwd_stages & MOE_STAGES_FWD != MOE_STAGES_FWD:
            raise ValueError("experts4: both products at once, in its own x_form: no mx and no other fwd_stages")
        if experts4.k != buf.k:   # the products divide src_of by it
            raise ValueError(f"experts4: made for k = {experts4.k}, the buffers for k = {buf.k}")
    _check_losses(router, routing)
    x_in = x
    if norms is not None:
        x = norms[0].before(x_in, norms[1])
    if router is not None:
        logits = router[0].project(x, router[1])
    if routing is not None:
        moe_route_scores(logits, buf.k, buf.topk_idx, buf.topk_w, buf.counts, buf.offsets, buf.row_of, buf.src_of,
                         buf.err, buf.route_ws, routing)
    else:
        moe_route_counts(logits, buf.k, buf.topk_idx, buf.topk_w, buf.counts, buf.offsets, buf.row_of,
                         buf.src_of, buf.M_cap, buf.err, buf.route_ws, renorm)
    if router is not None:
        router[0].losses(buf.topk_idx)
    buf.xt_from_forward = bool(mx)
    buf.served = experts4 is not None
    if experts4 is not None:
        experts4.forward(x, buf.offsets, buf.counts, buf.src_of, buf.a, buf.y)
    elif mx:
        if gather:
            raise ValueError("the MXFP8 FC1 reads the quantized permuted copy: no row gather")
        # X_perm only as its MXFP8 copies: row-wise (FC1) and column-wise (FC1 wgrad)
        moe_permute_quant_mxfp8(x, buf.src_of, buf.k, buf.E, MOE_QUANT_ROWWISE | MOE_QUANT_COLWISE,
                                buf.x_q, buf.x_s, buf.xt_q, buf.xt_s)
        moe_grouped_mlp_fwd(None, w1, w2, buf.offsets, buf.h if store_h else None, buf.a,
                            buf.y, fwd_stages, mx=buf.mx_fwd(), act=act)
    elif gather:
        moe_grouped_mlp_fwd(x, w1, w2, buf.offsets, buf.h if store_h else None, buf.a, buf.y,
                            fwd_stages | MOE_GATHER_ROWS, act=act, src_of=buf.src_of, k=buf.k)
    else:
        moe_permute(x, buf.row_of, buf.src_of, buf.offsets, buf.k, buf.E, buf.x_perm)
        moe_grouped_mlp_fwd(buf.x_perm, w1, w2, buf.offsets, buf.h if store_h else None, buf.a,
                            buf.y, fwd_stages, act=act)
    if buf.ckpt8 and store_h and (fwd_stages & MOE_STAGE_FC1) and experts4 is None:
        moe_quant_mxfp8(buf.h, MOE_QUANT_ROWWISE, buf.h_q, buf.h_s)
    if norms is not None and shared is None:   # the combination is the post norm's first step
        norms[0].after(x_in, *norms[2:], buf.y, row_of=buf.row_of, topk_w=buf.topk_w, total=buf.out)
        return
    moe_combine(buf.y, buf.row_of, buf.topk_w, buf.k, buf.out)
    if shared is not None:
        shared[0].forward(x, *shared[1:], buf.out)
    if norms is not None:
        norms[0].after(x_in, *norms[2:], buf.out)


def backward(buf: Buffers, dout, w1, w2, stages=MOE_STAGES_BWD, act=MOE_ACT_SWIGLU, logits=None,
             renorm=False, x=None, mx=False, dgrad2_mx=True, mx_bf16_copies=True, router=None, shared=None,
             x_tokens=None, routing=None, norms=None):
    """gather dO -> dgrad2+dGLU (+dS) -> wgrad2 -> dgrad1 -> unpermute-sum -> wgrad1, and with
    the forward's logits also the router backward dS -> dlogits. With x given (the un-permuted
    input), the GEMMs read x and dO through src_of instead of permuted copies. With mx (buffers
    made with mx=True and quantize_weights done), dY_u is quantized (row-wise for the FC2 dgrad
    when dgrad2_mx, column-wise for the FC2 wgrad), X_perm column-wise unless the MXFP8 forward
    already did, and the GEMMs run on MXFP8 (the FC2 dgrad only with dgrad2_mx). With mx and
    mx_bf16_copies=False the FC2 dgrad writes only the MXFP8 copies of dH and A' (buf.dh and
    buf.a_w are left untouched), which is all the later MXFP8 stages read. The FC1 wgrad runs
    last, after the unpermute-sum has read dX_perm. router and shared as in forward (x_tokens:
    the layer's input x [T, d] for their weight gradients, unless x is given or they keep an 8-bit
    checkpoint of it): their gradients are added to dx. routing as in forward. norms as in forward, with x or
    x_tokens the residual stream that it was given: dout is the gradient of the block's output, and the BlockNorms' dx
    that of the residual stream."""
    if buf.served:
        raise ValueError("the last forward ran on 4-bit weights and kept nothing for a backward pass")
    _check_losses(router, routing)
    x_in = x if x is not None else x_tokens
    if norms is not None:
        if x_in is None:
            raise ValueError("the norms' backward needs x or x_tokens")
        stream, dblock = x_in, dout
        dout = norms[0].back_after(dblock, *norms[2:], buf.out)
        x_in = norms[0].y
        x = x_in if x is not None else None
    if x_in is None and (router is not None or (shared is not None and not shared[0].x8)):
        raise ValueError("the router's and the shared expert's weight gradients need x or x_tokens")
    if buf.ckpt8 and (stages & MOE_STAGE_DGRAD2):
        moe_dequant_mxfp8(buf.h_q, buf.h_s, buf.h)
    early, late = stages & ~MOE_STAGE_WGRAD1, stages & MOE_STAGE_WGRAD1
    if mx:
        if x is not None:
            raise ValueError("the MXFP8 backward quantizes the permuted copies: no row gather")
        if dgrad2_mx:   # dY_u only as its MXFP8 copies
            moe_permute_quant_mxfp8(dout, buf.src_of, buf.k, buf.E, MOE_QUANT_ROWWISE | MOE_QUANT_COLWISE,
                                    buf.dy_q, buf.dy_s, buf.dyt_q, buf.dyt_s)
        else:
            moe_permute(dout, buf.row_of, buf.src_of, buf.offsets, buf.k, buf.E, buf.dy_u)
            moe_quant_mxfp8(buf.dy_u, MOE_QUANT_COLWISE, None, None, buf.dyt_q, buf.dyt_s)
        if not buf.xt_from_forward:
            moe_quant_mxfp8(buf.x_perm, MOE_QUANT_COLWISE, None, None, buf.xt_q, buf.xt_s)
        dh, a_w = (buf.dh, buf.a_w) if mx_bf16_copies else (None, None)
        bwd = lambda st: moe_grouped_mlp_bwd(buf.x_perm, w1, w2, buf.h, buf.dy_u, buf.topk_w, buf.src_of,
                                             buf.row_of, buf.offsets, dh, a_w, buf.ds, buf.dx_perm, buf.dw1,
                                             buf.dw2, buf.bwd_ws, st, act=act, mx=buf.mx_bwd(dgrad2_mx))
    elif x is not None:
        bwd = lambda st: moe_grouped_mlp_bwd(x, w1, w2, buf.h, dout, buf.topk_w, buf.src_of, buf.row_of,
                                             buf.offsets, buf.dh, buf.a_w, buf.ds, buf.dx_perm, buf.dw1,
                                             buf.dw2, buf.bwd_ws, st | MOE_GATHER_ROWS, act=act)
    else:
        moe_permute(dout, buf.row_of, buf.src_of, buf.offsets, buf.k, buf.E, buf.dy_u)
        bwd = lambda st: moe_grouped_mlp_bwd(buf.x_perm, w1, w2, buf.h, buf.dy_u, buf.topk_w, buf.src_of,
                                             buf.row_of, buf.offsets, buf.dh, buf.a_w, buf.ds, buf.dx_perm,
                                             buf.dw1, buf.dw2, buf.bwd_ws, st, act=act)
    if early:
        bwd(early)
    moe_combine(buf.dx_perm, buf.row_of, None, buf.k, buf.dx)
    if late:
        bwd(late)
    if shared is not None:
        shared[0].backward(x_in, dout, *shared[1:], buf.dx)
    if router is not None:
        logits = router[0].logits
    if logits is not None:
        if routing is not None:
            moe_route_scores_bwd(logits, buf.topk_idx, buf.ds, buf.dlogits, routing)
        else:
            moe_route_bwd(logits, buf.topk_idx, buf.ds, buf.dlogits, renorm)
    if router is not None:
        router[0].backward(x_in, router[1], buf.dlogits, buf.dx)
    if norms is not None:
        norms[0].back_before(buf.dx, dblock, stream, norms[1])
