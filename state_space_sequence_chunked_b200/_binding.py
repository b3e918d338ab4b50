"""ctypes binding of libssd (include/ssd.h): argument marshalling only.

Every step of the computation runs in the CUDA library. Torch tensors supply
device memory and the current CUDA stream. If the library is missing the calls
raise; there is no other implementation behind them.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
STATUS = {0: "SSD_OK", 1: "SSD_ERR_INVALID_ARG", 2: "SSD_ERR_UNSUPPORTED", 3: "SSD_ERR_ALIGNMENT",
          4: "SSD_ERR_WORKSPACE", 5: "SSD_ERR_CUDA", 6: "SSD_ERR_TIMEOUT"}


class SSDError(RuntimeError):
    def __init__(self, status: int, fn: str, text: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({text})")
        self.status = status
        self.name = STATUS.get(status, str(status))


class ShapeT(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seqlen", "nheads", "headdim", "ngroups", "dstate")]


class PlanT(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("kernels", ctypes.c_int32), ("workspace_bytes", ctypes.c_size_t)]


PATHS = {0: "none", 1: "simt", 2: "tcgen05", 3: "mma"}

_lib = None
_vp, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "ssd_strerror": ([ctypes.c_int], ctypes.c_char_p),
    "ssd_fwd_workspace_bytes": ([ctypes.POINTER(ShapeT), ctypes.c_int, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "ssd_fwd_plan": ([ctypes.POINTER(ShapeT), ctypes.c_int, _i64, ctypes.POINTER(PlanT)], ctypes.c_int),
    "ssd_fwd": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 7 + [_i64, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    "ssd_fwd_static_scratch": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 7 + [_i64, _vp, _vp, _vp], ctypes.c_int),
    "ssd_fwd_status": ([ctypes.POINTER(ShapeT), ctypes.c_int, _i64, _vp, _vp], ctypes.c_int),
    "ssd_set_wait_limit_us": ([ctypes.c_int32], ctypes.c_int),
    "ssd_verify": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 7 + [_i64, _vp, _vp, _vp], ctypes.c_int),
    "ssd_select_state": ([ctypes.POINTER(ShapeT), _i64] + [_vp] * 5, ctypes.c_int),
    "ssd_advance_state": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 5 + [_i64, _vp, _vp, _vp], ctypes.c_int),
    "ssd_decode_step": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 9, ctypes.c_int),
    "ssd_cp_decay": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 5, ctypes.c_int),
    "ssd_cp_combine": ([ctypes.POINTER(ShapeT), _i64, _i64] + [_vp] * 5, ctypes.c_int),
    "ssd_cp_correct": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 8, ctypes.c_int),
    "ssd_bwd_workspace_bytes": ([ctypes.POINTER(ShapeT), ctypes.c_int, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "ssd_bwd_plan": ([ctypes.POINTER(ShapeT), ctypes.c_int, _i64, ctypes.POINTER(PlanT)], ctypes.c_int),
    "ssd_conv_split": ([ctypes.POINTER(ShapeT), ctypes.c_int, _vp, _i64, _vp, _i64, _vp, _vp, _i64] + [_vp] * 6,
                       ctypes.c_int),
    "ssd_gated_rmsnorm": ([_i64, _i64, _i64, ctypes.c_int, _vp, _vp, _i64, _vp, ctypes.c_float, _vp, _vp],
                          ctypes.c_int),
    "ssd_bwd": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 7 + [_i64] + [_vp] * 9 + [_vp, _sz, _vp],
                ctypes.c_int),
    "ssd_delta_fwd_plan": ([ctypes.POINTER(ShapeT), ctypes.c_int, ctypes.POINTER(PlanT)], ctypes.c_int),
    "ssd_delta_fwd": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 9 + [_sz, _vp], ctypes.c_int),
    "ssd_delta_status": ([ctypes.POINTER(ShapeT), ctypes.c_int, _vp, _vp], ctypes.c_int),
    "ssd_delta_decode_step": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 9, ctypes.c_int),
    "ssd_delta_bwd_plan": ([ctypes.POINTER(ShapeT), ctypes.c_int, ctypes.POINTER(PlanT)], ctypes.c_int),
    "ssd_delta_bwd": ([ctypes.POINTER(ShapeT), ctypes.c_int] + [_vp] * 15 + [_sz, _vp], ctypes.c_int),
    "ssd_norm_bwd_workspace_bytes": ([_i64, _i64, ctypes.POINTER(_sz)], ctypes.c_int),
    "ssd_add_rmsnorm": ([_i64, _i64, ctypes.c_int, ctypes.c_int] + [_vp] * 4 + [ctypes.c_float] + [_vp] * 3, ctypes.c_int),
    "ssd_add_rmsnorm_bwd": ([_i64, _i64, ctypes.c_int, ctypes.c_int, _vp, _vp, ctypes.c_float] + [_vp] * 9 + [_sz, _vp],
                            ctypes.c_int),
    "ssd_norm_gate": ([_i64, _i64, _i64, ctypes.c_int, _vp, _vp, _i64, _vp, ctypes.c_float, _vp, _vp], ctypes.c_int),
    "ssd_norm_gate_bwd": ([_i64, _i64, _i64, ctypes.c_int, _vp, _vp, _i64, _vp, ctypes.c_float, _vp, _vp, _vp, _i64, _vp,
                           _vp, _sz, _vp], ctypes.c_int),
    "ssd_gated_rmsnorm_bwd": ([_i64, _i64, _i64, ctypes.c_int, _vp, _vp, _i64, _vp, ctypes.c_float, _vp, _vp, _vp, _i64, _vp,
                               _vp, _sz, _vp], ctypes.c_int),
}

CP_BLOCK = 128  # SSD_CP_BLOCK: tokens per decay block


def lib():
    """Load libssd.so (built in-tree by state_space_sequence_chunked_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libssd.so is not built ({LIB_PATH}); run state_space_sequence_chunked_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def _check(status: int, fn: str):
    if status != 0:
        raise SSDError(status, fn, lib().ssd_strerror(status).decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SSD_F32
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libssd takes CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("libssd takes contiguous tensors")
        dev = t.device if dev is None else dev
    return dev


def _dev_rows(dev, *ts):
    """Row views (a column slice of wider rows): CUDA, on `dev`, unit column stride, rows at one
    stride (the C calls take that stride)."""
    for t in ts:
        if not t.is_cuda or (dev is not None and t.device != dev):
            raise ValueError("libssd takes CUDA tensors on one device")
        if t.stride(-1) != 1 or any(t.stride(i) != t.stride(i + 1) * t.shape[i + 1] for i in range(t.dim() - 2)):
            raise ValueError("row views need unit column stride and evenly spaced rows")


def _stream(dev, stream):
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    return ctypes.c_void_p(stream.cuda_stream)


def fwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, dtype_code, chunk) -> int:
    shape = ShapeT(batch, seqlen, nheads, headdim, ngroups, dstate)
    out = _sz(0)
    _check(lib().ssd_fwd_workspace_bytes(ctypes.byref(shape), dtype_code, chunk, ctypes.byref(out)),
           "ssd_fwd_workspace_bytes")
    return out.value


def fwd_plan(batch, seqlen, nheads, headdim, ngroups, dstate, dtype_code, chunk) -> dict:
    """{'path': 'simt'|'tcgen05'|'none', 'kernels': launches per call, 'workspace_bytes': int}."""
    shape = ShapeT(batch, seqlen, nheads, headdim, ngroups, dstate)
    out = PlanT()
    _check(lib().ssd_fwd_plan(ctypes.byref(shape), dtype_code, chunk, ctypes.byref(out)), "ssd_fwd_plan")
    return {"path": PATHS.get(out.path, str(out.path)), "kernels": out.kernels,
            "workspace_bytes": out.workspace_bytes}


def ssd_fwd(x, dt, A, B, C, D=None, h0=None, *, chunk: int, y=None, h_final=None,
            return_final_state: bool = True, workspace=None, stream=None, check: bool = False):
    """y, h_final = ssd_fwd(x [B,L,H,P], dt [B,L,H], A [H] f32, B/C [B,L,G,N], D [H] f32?, h0 [B,H,P,N] f32?).

    check=True synchronizes the stream after the launch and raises SSDError (SSD_ERR_TIMEOUT)
    if a bounded device-side wait ran out, which leaves y and h_final incomplete."""
    dev = _dev(x, dt, A, B, C, D, h0, y, h_final, workspace)
    Bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(x)
    shape = ShapeT(Bsz, L, H, P, G, N)
    if y is None:
        y = torch.empty_like(x)
    if h_final is None and return_final_state:
        h_final = torch.empty((Bsz, H, P, N), dtype=torch.float32, device=dev)
    need = fwd_workspace_bytes(Bsz, L, H, P, G, N, code, chunk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ssd_fwd(ctypes.byref(shape), code, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                       _ptr(h0), chunk, _ptr(y), _ptr(h_final), _ptr(workspace), ws_bytes,
                       _stream(dev, stream))
    _check(st, "ssd_fwd")
    if check:
        _check(lib().ssd_fwd_status(ctypes.byref(shape), code, chunk, _ptr(workspace), _stream(dev, stream)),
               "ssd_fwd")
    return y, h_final


def fwd_status(shape_args, dtype_code, chunk, workspace, stream=None) -> int:
    """Raw ssd_fwd_status code for the last ssd_fwd on `workspace` (synchronizes the stream).

    shape_args = (batch, seqlen, nheads, headdim, ngroups, dstate)."""
    shape = ShapeT(*shape_args)
    dev = workspace.device if workspace is not None else torch.device("cuda", torch.cuda.current_device())
    return lib().ssd_fwd_status(ctypes.byref(shape), dtype_code, chunk, _ptr(workspace), _stream(dev, stream))


def set_wait_limit_us(us: int):
    """Test hook: limit of every bounded device-side wait in later launches (0: the built-in 2 s)."""
    _check(lib().ssd_set_wait_limit_us(int(us)), "ssd_set_wait_limit_us")


def ssd_verify(h0, x, dt, A, B, C, D=None, *, states_out=None, y=None, return_states: bool = True,
               stream=None):
    """y [B,K,H,P], states_out [B,K,H,P,N] = ssd_verify(h0 [B,H,P,N] f32, x [B,K,H,P], dt, A, B, C, D).

    return_states=False (and no states_out given) writes y only; states_out is then None."""
    dev = _dev(h0, x, dt, A, B, C, D, states_out, y)
    Bsz, K, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    shape = ShapeT(Bsz, K, H, P, G, N)
    if y is None:
        y = torch.empty_like(x)
    if states_out is None and return_states:
        states_out = torch.empty((Bsz, K, H, P, N), dtype=torch.float32, device=dev)
    st = lib().ssd_verify(ctypes.byref(shape), _dtype_code(x), _ptr(h0), _ptr(x), _ptr(dt), _ptr(A), _ptr(B),
                          _ptr(C), _ptr(D), K, _ptr(states_out), _ptr(y), _stream(dev, stream))
    _check(st, "ssd_verify")
    return y, states_out


def ssd_select_state(h0, states_out, accepted, *, h_keep=None, stream=None):
    """h_keep[b] = h0[b] if accepted[b] == 0 else states_out[b, accepted[b] - 1] (bit-exact)."""
    dev = _dev(h0, states_out, accepted, h_keep)
    Bsz, K, H, P, N = states_out.shape
    if accepted.dtype != torch.int32:
        raise TypeError("accepted must be int32")
    shape = ShapeT(Bsz, K, H, P, 1, N)
    if h_keep is None:
        h_keep = torch.empty_like(h0)
    st = lib().ssd_select_state(ctypes.byref(shape), K, _ptr(h0), _ptr(states_out), _ptr(accepted),
                                _ptr(h_keep), _stream(dev, stream))
    _check(st, "ssd_select_state")
    return h_keep


def ssd_advance_state(h0, x, dt, A, B, accepted, *, h_keep=None, stream=None):
    """h_keep[b] = state after the first accepted[b] draft tokens from h0[b] (h_keep may be h0: in place)."""
    dev = _dev(h0, x, dt, A, B, accepted, h_keep)
    if accepted.dtype != torch.int32:
        raise TypeError("accepted must be int32")
    Bsz, K, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    shape = ShapeT(Bsz, K, H, P, G, N)
    if h_keep is None:
        h_keep = torch.empty_like(h0)
    st = lib().ssd_advance_state(ctypes.byref(shape), _dtype_code(x), _ptr(h0), _ptr(x), _ptr(dt), _ptr(A),
                                 _ptr(B), K, _ptr(accepted), _ptr(h_keep), _stream(dev, stream))
    _check(st, "ssd_advance_state")
    return h_keep


def ssd_decode_step(state, x, dt, A, B, C, D=None, *, y=None, stream=None):
    """One token in place: state [B,H,P,N] f32 <- exp(dt A) state + dt x B^T; returns y [B,H,P] = state C + D x.
    x [B,H,P], dt [B,H], B/C [B,G,N]."""
    dev = _dev(state, x, dt, A, B, C, D, y)
    Bsz, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    shape = ShapeT(Bsz, 1, H, P, G, N)
    if y is None:
        y = torch.empty_like(x)
    st = lib().ssd_decode_step(ctypes.byref(shape), _dtype_code(x), _ptr(state), _ptr(x), _ptr(dt), _ptr(A),
                               _ptr(B), _ptr(C), _ptr(D), _ptr(y), _stream(dev, stream))
    _check(st, "ssd_decode_step")
    return y


def ssd_cp_decay(dt, A, *, block_decay=None, total=None, stream=None):
    """block_decay [B,H,ceil(L/128)], total [B,H] = sums of dt*A over a segment's blocks and over the segment."""
    dev = _dev(dt, A, block_decay, total)
    Bsz, L, H = dt.shape
    nblk = (L + CP_BLOCK - 1) // CP_BLOCK
    if block_decay is None:
        block_decay = torch.empty((Bsz, H, max(nblk, 1)), dtype=torch.float32, device=dev)
    if total is None:
        total = torch.empty((Bsz, H), dtype=torch.float32, device=dev)
    shape = ShapeT(Bsz, L, H, 1, 1, 1)
    st = lib().ssd_cp_decay(ctypes.byref(shape), _dtype_code(dt), _ptr(dt), _ptr(A), _ptr(block_decay), _ptr(total),
                            _stream(dev, stream))
    _check(st, "ssd_cp_decay")
    return block_decay, total


def ssd_cp_combine(states, totals, rank, *, s_in=None, h_final=None, want_final=True, stream=None):
    """s_in (state entering segment `rank`), h_final (its true end state) from the gathered
    states [R,B,H,P,N] and totals [R,B,H]."""
    dev = _dev(states, totals, s_in, h_final)
    R, Bsz, H, P, N = states.shape
    if s_in is None:
        s_in = torch.empty((Bsz, H, P, N), dtype=torch.float32, device=dev)
    if h_final is None and want_final:
        h_final = torch.empty((Bsz, H, P, N), dtype=torch.float32, device=dev)
    shape = ShapeT(Bsz, 0, H, P, 1, N)
    st = lib().ssd_cp_combine(ctypes.byref(shape), R, rank, _ptr(states), _ptr(totals), _ptr(s_in), _ptr(h_final),
                              _stream(dev, stream))
    _check(st, "ssd_cp_combine")
    return s_in, h_final


def ssd_cp_correct(dt, A, C, block_decay, s_in, y, *, status=None, stream=None):
    """y += exp(cumulative dt*A from the segment start) * C S_in^T, in place; returns y.
    status: optional int32 device tensor (one element, zeroed by the caller); bit 0 is set if a
    bounded device-side wait ran out."""
    dev = _dev(dt, A, C, block_decay, s_in, y, status)
    Bsz, L, H, P = y.shape
    G, N = C.shape[2], C.shape[3]
    shape = ShapeT(Bsz, L, H, P, G, N)
    st = lib().ssd_cp_correct(ctypes.byref(shape), _dtype_code(y), _ptr(dt), _ptr(A), _ptr(C), _ptr(block_decay),
                              _ptr(s_in), _ptr(y), _ptr(status), _stream(dev, stream))
    _check(st, "ssd_cp_correct")
    return y


def bwd_workspace_bytes(batch, seqlen, nheads, headdim, ngroups, dstate, dtype_code, chunk) -> int:
    shape = ShapeT(batch, seqlen, nheads, headdim, ngroups, dstate)
    out = _sz(0)
    _check(lib().ssd_bwd_workspace_bytes(ctypes.byref(shape), dtype_code, chunk, ctypes.byref(out)),
           "ssd_bwd_workspace_bytes")
    return out.value


def bwd_plan(batch, seqlen, nheads, headdim, ngroups, dstate, dtype_code, chunk) -> dict:
    """{'path': 'simt'|'mma'|'none', 'kernels': launches per call, 'workspace_bytes': int}."""
    shape = ShapeT(batch, seqlen, nheads, headdim, ngroups, dstate)
    out = PlanT()
    _check(lib().ssd_bwd_plan(ctypes.byref(shape), dtype_code, chunk, ctypes.byref(out)), "ssd_bwd_plan")
    return {"path": PATHS.get(out.path, str(out.path)), "kernels": out.kernels,
            "workspace_bytes": out.workspace_bytes}


def ssd_bwd(x, dt, A, B, C, D, h0, dy, dh_final=None, *, chunk: int, want_dD: bool = True,
            want_dh0: bool = True, out=None, workspace=None, stream=None):
    """Gradients of sum(dy * y) + sum(dh_final * h_final) through ssd_fwd.

    Returns a dict dx, ddt, dA, dB, dC, dD (None unless want_dD), dh0 (None unless want_dh0);
    `out` may supply any of those tensors to write into."""
    dev = _dev(x, dt, A, B, C, D, h0, dy, dh_final, workspace)
    Bsz, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(x)
    shape = ShapeT(Bsz, L, H, P, G, N)
    o = dict(out or {})
    o.setdefault("dx", torch.empty_like(x))
    o.setdefault("ddt", torch.empty_like(dt))
    o.setdefault("dA", torch.empty(H, dtype=torch.float32, device=dev))
    o.setdefault("dB", torch.empty_like(B))
    o.setdefault("dC", torch.empty_like(C))
    o.setdefault("dD", torch.empty(H, dtype=torch.float32, device=dev) if want_dD else None)
    o.setdefault("dh0", torch.empty((Bsz, H, P, N), dtype=torch.float32, device=dev) if want_dh0 else None)
    need = bwd_workspace_bytes(Bsz, L, H, P, G, N, code, chunk)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ssd_bwd(ctypes.byref(shape), code, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                       _ptr(h0), chunk, _ptr(dy), _ptr(dh_final), _ptr(o["dx"]), _ptr(o["ddt"]), _ptr(o["dA"]),
                       _ptr(o["dB"]), _ptr(o["dC"]), _ptr(o["dD"]), _ptr(o["dh0"]), _ptr(workspace), ws_bytes,
                       _stream(dev, stream))
    _check(st, "ssd_bwd")
    return o


def ssd_conv_split(xbc, dt_raw, conv_w, conv_b, dt_bias, *, nheads, headdim, ngroups, dstate, out=None,
                   stream=None):
    """x [B,L,H,P], B, C [B,L,G,N], dt [B,L,H] from the convolution + SiLU of the x B C channels and
    softplus(dt_raw + dt_bias). xbc and dt_raw are [B, L, *] views with unit column stride (the
    input projection's columns can be passed in place)."""
    dev = _dev(conv_w, conv_b, dt_bias)
    _dev_rows(dev, xbc, dt_raw)
    Bsz, L = xbc.shape[0], xbc.shape[1]
    H, P, G, N = nheads, headdim, ngroups, dstate
    assert xbc.stride(2) == 1 and dt_raw.stride(2) == 1 and xbc.stride(0) == L * xbc.stride(1)
    assert dt_raw.stride(0) == L * dt_raw.stride(1)
    code = _dtype_code(xbc)
    o = dict(out or {})
    o.setdefault("x", torch.empty(Bsz, L, H, P, dtype=xbc.dtype, device=dev))
    o.setdefault("B", torch.empty(Bsz, L, G, N, dtype=xbc.dtype, device=dev))
    o.setdefault("C", torch.empty(Bsz, L, G, N, dtype=xbc.dtype, device=dev))
    o.setdefault("dt", torch.empty(Bsz, L, H, dtype=xbc.dtype, device=dev))
    shape = ShapeT(Bsz, L, H, P, G, N)
    st = lib().ssd_conv_split(ctypes.byref(shape), code, _ptr(xbc), xbc.stride(1), _ptr(dt_raw), dt_raw.stride(1),
                              _ptr(conv_w), _ptr(conv_b), conv_w.shape[1], _ptr(dt_bias), _ptr(o["x"]), _ptr(o["B"]),
                              _ptr(o["C"]), _ptr(o["dt"]), _stream(dev, stream))
    _check(st, "ssd_conv_split")
    return o


def ssd_gated_rmsnorm(y, z, weight, *, ngroups, eps=1e-5, out=None, stream=None):
    """out = weight * RMSNorm over `ngroups` groups of (y * silu(z)); y [..., dim] contiguous,
    z [..., dim] with unit column stride (a column slice of a wider row is fine)."""
    dev = _dev(y, weight, out)
    _dev_rows(dev, z)
    dim = y.shape[-1]
    rows = y.numel() // dim if dim else 0
    assert z.stride(-1) == 1
    zs = z.stride(-2) if z.dim() >= 2 else dim
    if out is None:
        out = torch.empty_like(y)
    st = lib().ssd_gated_rmsnorm(rows, dim, ngroups, _dtype_code(y), _ptr(y), _ptr(z), zs, _ptr(weight), float(eps),
                                 _ptr(out), _stream(dev, stream))
    _check(st, "ssd_gated_rmsnorm")
    return out



# ---- the gated delta rule and the norms around its block ------------------------------


def _need(name, t, shape, dtype, dev):
    """t (None passes) has this shape and type, is contiguous and on `dev` (a CUDA device's index)."""
    if t is None or (t.get_device() == dev >= 0 and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        return
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name}: libssd takes CUDA tensors on one device (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: libssd takes contiguous tensors")


class _On:
    """The calls within run with device `dev` current and allocate on `stream` (None: the device's
    current stream), so that memory freed afterwards is not handed out again before the kernels are
    done. Enters with the stream's handle."""

    __slots__ = ("dev", "stream", "ctx")

    def __init__(self, dev, stream):
        self.dev, self.stream, self.ctx = dev, stream, None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device.index != self.dev:
                raise ValueError("stream: of another device than the tensors")
            self.ctx = torch.cuda.stream(self.stream)
        elif self.dev != torch.cuda.current_device():
            self.ctx = torch.cuda.device(self.dev)
        if self.ctx is not None:
            self.ctx.__enter__()
        if self.stream is not None:
            return self.stream.cuda_stream
        return _raw_stream(self.dev)

    def __exit__(self, *e):
        if self.ctx is not None:
            self.ctx.__exit__(*e)


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# the handle alone where torch offers it: a fifteenth of the time, and it counts for single tokens
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _at(t):
    return None if t is None else t.data_ptr()


def _delta_shape(x, g, beta, B, C, batched):
    """(ShapeT, dtype code) of the delta rule's inputs, checked against one another."""
    xs, bs, gs, dev, dt = x.shape, B.shape, g.shape, x.get_device(), x.dtype
    # all in one expression: for single tokens the checks cost as much as the launch
    if not (len(xs) == len(bs) == (4 if batched else 3) and xs[:-2] == bs[:-2] and gs == xs[:-1] and beta.shape == gs
            and C.shape == bs and dev >= 0 and g.get_device() == dev and beta.get_device() == dev and B.get_device() == dev
            and C.get_device() == dev and g.dtype is dt and beta.dtype is dt and B.dtype is dt and C.dtype is dt
            and x.is_contiguous() and g.is_contiguous() and beta.is_contiguous() and B.is_contiguous() and C.is_contiguous()):
        if len(xs) != (4 if batched else 3) or len(bs) != len(xs):
            raise ValueError("x and B: wrong number of dimensions")
        for name, t, shape in (("x", x, xs), ("g", g, xs[:-1]), ("beta", beta, xs[:-1]), ("B", B, (*xs[:-2], *bs[-2:])),
                               ("C", C, (*xs[:-2], *bs[-2:]))):
            _need(name, t, torch.Size(shape), dt, dev)
        raise ValueError("x, g, beta, B, C do not fit one another")
    return ShapeT(xs[0], xs[1] if batched else 1, xs[-2], xs[-1], bs[-2], bs[-1]), _dtype_code(x)


def _delta_plan(fn, shape, code):
    out = PlanT()
    _check(getattr(lib(), fn)(ctypes.byref(shape), code, ctypes.byref(out)), fn)
    return out


def delta_fwd_plan(batch, seqlen, nheads, headdim, ngroups, dstate, dtype_code) -> dict:
    """{'path': 'simt'|'tcgen05'|'none', 'kernels': launches per call, 'workspace_bytes': int}."""
    out = _delta_plan("ssd_delta_fwd_plan", ShapeT(batch, seqlen, nheads, headdim, ngroups, dstate), dtype_code)
    return {"path": PATHS.get(out.path, str(out.path)), "kernels": out.kernels, "workspace_bytes": out.workspace_bytes}


def delta_bwd_plan(batch, seqlen, nheads, headdim, ngroups, dstate, dtype_code) -> dict:
    """As delta_fwd_plan, of ssd_delta_bwd."""
    out = _delta_plan("ssd_delta_bwd_plan", ShapeT(batch, seqlen, nheads, headdim, ngroups, dstate), dtype_code)
    return {"path": PATHS.get(out.path, str(out.path)), "kernels": out.kernels, "workspace_bytes": out.workspace_bytes}


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the inputs' device")
    return workspace


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def ssd_delta_fwd(x, g, beta, B, C, h0=None, *, y=None, h_final=None, return_final_state: bool = True, workspace=None,
                  stream=None):
    """y, h_final of the gated delta rule: x [B,L,H,P], g (log decay) and beta [B,L,H], B (keys) and
    C (queries) [B,L,G,N], h0 [B,H,P,N] f32."""
    shape, code = _delta_shape(x, g, beta, B, C, True)
    dev = x.get_device()
    state = (x.shape[0], *x.shape[2:], B.shape[-1])
    _need("h0", h0, state, torch.float32, dev)
    _need("y", y, x.shape, x.dtype, dev)
    _need("h_final", h_final, state, torch.float32, dev)
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x)
        if h_final is None and return_final_state:
            h_final = torch.empty(state, dtype=torch.float32, device=dev)
        ws = _workspace(workspace, _delta_plan("ssd_delta_fwd_plan", shape, code).workspace_bytes, dev)
        _check(lib().ssd_delta_fwd(ctypes.byref(shape), code, _at(x), _at(g), _at(beta), _at(B), _at(C), _at(h0),
                                   _at(y), _at(h_final), _at(ws), _bytes(ws), st), "ssd_delta_fwd")
    return y, h_final


def delta_status(shape_args, dtype_code, workspace, stream=None) -> int:
    """Raw ssd_delta_status code for the last ssd_delta_fwd or ssd_delta_bwd on `workspace`
    (synchronizes the stream). shape_args = (batch, seqlen, nheads, headdim, ngroups, dstate)."""
    dev = workspace.get_device() if workspace is not None else torch.cuda.current_device()
    with _On(dev, stream) as st:
        return lib().ssd_delta_status(ctypes.byref(ShapeT(*shape_args)), dtype_code, _at(workspace), st)


def ssd_delta_decode_step(state, x, g, beta, B, C, *, state_out=None, y=None, stream=None):
    """y [B,H,P] of one token of the gated delta rule; x [B,H,P], g and beta [B,H], B, C [B,G,N]. The
    state [B,H,P,N] f32 is updated in place, or left alone and the new one written to state_out."""
    shape, code = _delta_shape(x, g, beta, B, C, False)
    dev = x.get_device()
    size = (*x.shape, B.shape[-1])
    _need("state", state, size, torch.float32, dev)
    _need("state_out", state_out, size, torch.float32, dev)
    _need("y", y, x.shape, x.dtype, dev)
    with _On(dev, stream) as st:
        if y is None:
            y = torch.empty_like(x)
        _check(lib().ssd_delta_decode_step(ctypes.byref(shape), code, _at(state),
                                           _at(state if state_out is None else state_out), _at(x), _at(g), _at(beta),
                                           _at(B), _at(C), _at(y), st), "ssd_delta_decode_step")
    return y


def ssd_delta_bwd(x, g, beta, B, C, h0, dy, dh_final=None, *, want_dh0: bool = True, out=None, workspace=None, stream=None):
    """Gradients of sum(dy * y) + sum(dh_final * h_final) through ssd_delta_fwd.

    Returns a dict dx, dg, dbeta, dB, dC, dh0 (None unless want_dh0); `out` may supply any of those
    tensors to write into."""
    shape, code = _delta_shape(x, g, beta, B, C, True)
    dev = x.get_device()
    state = (x.shape[0], *x.shape[2:], B.shape[-1])
    _need("h0", h0, state, torch.float32, dev)
    _need("dy", dy, x.shape, x.dtype, dev)
    _need("dh_final", dh_final, state, torch.float32, dev)
    o = dict(out or {})
    with _On(dev, stream) as st:
        for name, like in (("dx", x), ("dg", g), ("dbeta", beta), ("dB", B), ("dC", C)):
            _need(name, o.get(name), like.shape, like.dtype, dev)
            if o.get(name) is None:
                o[name] = torch.empty_like(like)
        _need("dh0", o.get("dh0"), state, torch.float32, dev)
        if o.get("dh0") is None:
            o["dh0"] = torch.empty(state, dtype=torch.float32, device=dev) if want_dh0 else None
        ws = _workspace(workspace, _delta_plan("ssd_delta_bwd_plan", shape, code).workspace_bytes, dev)
        _check(lib().ssd_delta_bwd(ctypes.byref(shape), code, _at(x), _at(g), _at(beta), _at(B), _at(C), _at(h0),
                                   _at(dy), _at(dh_final), _at(o["dx"]), _at(o["dg"]), _at(o["dbeta"]), _at(o["dB"]),
                                   _at(o["dC"]), _at(o["dh0"]), _at(ws), _bytes(ws), st), "ssd_delta_bwd")
    return o


def norm_bwd_workspace_bytes(rows, dim) -> int:
    out = _sz(0)
    _check(lib().ssd_norm_bwd_workspace_bytes(rows, dim, ctypes.byref(out)), "ssd_norm_bwd_workspace_bytes")
    return out.value


def ssd_add_rmsnorm(x, residual, weight, *, scale=None, eps=1e-5, res_out=None, out=None, want_res: bool = True, stream=None):
    """res, out: r = residual + scale * x and weight * r / sqrt(mean(r^2) + eps) over the last axis.

    residual (None = 0) is in x's type or fp32, weight and scale (None = 1) are fp32. res_out may be
    residual itself. want_res=False (and no res_out given) returns None for r."""
    dev, dim = x.get_device(), x.shape[-1] if x.dim() else 0
    like = next((t for t in (residual, res_out) if t is not None), x)
    rdt, code, rcode = like.dtype, _dtype_code(x), _dtype_code(like)  # (a type that the library lacks ends here)
    _need("x", x, x.shape, x.dtype, dev)
    _need("residual", residual, x.shape, rdt, dev)
    _need("weight", weight, (dim,), torch.float32, dev)
    _need("scale", scale, (dim,), torch.float32, dev)
    _need("res_out", res_out, x.shape, rdt, dev)
    _need("out", out, x.shape, x.dtype, dev)
    with _On(dev, stream) as st:
        if res_out is None and want_res:
            res_out = torch.empty(x.shape, dtype=rdt, device=dev)
        if out is None:
            out = torch.empty_like(x)
        _check(lib().ssd_add_rmsnorm(x.numel() // dim if dim else 0, dim, code, rcode, _at(x), _at(residual), _at(scale),
                                     _at(weight), float(eps), _at(res_out), _at(out), st), "ssd_add_rmsnorm")
    return res_out, out


def ssd_add_rmsnorm_bwd(res, weight, dout, dres_in=None, *, x=None, scale=None, eps=1e-5, want_dw: bool = True, out=None,
                        workspace=None, stream=None):
    """Gradients of ssd_add_rmsnorm from its r (`res`), the cotangent dout of out and dres_in of r.

    Returns a dict dres (the residual's), dx, dw (None unless want_dw), dscale (None unless scale and
    the forward's x are given); `out` may supply any of those tensors to write into (dres may be
    dres_in, dx may be dout)."""
    dev, dim = dout.get_device(), dout.shape[-1] if dout.dim() else 0
    code, rcode = _dtype_code(dout), _dtype_code(res)
    _need("dout", dout, dout.shape, dout.dtype, dev)
    _need("res", res, dout.shape, res.dtype, dev)
    _need("dres_in", dres_in, dout.shape, res.dtype, dev)
    _need("x", x, dout.shape, dout.dtype, dev)
    _need("weight", weight, (dim,), torch.float32, dev)
    _need("scale", scale, (dim,), torch.float32, dev)
    rows = dout.numel() // dim if dim else 0
    o = dict(out or {})
    with _On(dev, stream) as st:
        for name, dt, shape, want in (("dres", res.dtype, dout.shape, True), ("dx", dout.dtype, dout.shape, True),
                                      ("dw", torch.float32, (dim,), want_dw),
                                      ("dscale", torch.float32, (dim,), scale is not None and x is not None)):
            _need(name, o.get(name), shape, dt, dev)
            if o.get(name) is None:
                o[name] = torch.empty(shape, dtype=dt, device=dev) if want else None
        sums = o["dw"] is not None or o["dscale"] is not None
        ws = _workspace(workspace, norm_bwd_workspace_bytes(rows, dim) if sums else 0, dev)
        _check(lib().ssd_add_rmsnorm_bwd(rows, dim, code, rcode, _at(res), _at(weight), float(eps), _at(dout),
                                         _at(dres_in), _at(x), _at(scale), _at(o["dres"]), _at(o["dx"]), _at(o["dw"]),
                                         _at(o["dscale"]), _at(ws), _bytes(ws), st), "ssd_add_rmsnorm_bwd")
    return o


def _rows_view(name, t, like, dev):
    """The row stride of t [..., dim], a column slice of evenly spaced wider rows."""
    if t.get_device() != dev or t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError(f"{name}: expected {tuple(like.shape)} {like.dtype} on one device")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: row views need unit column stride")
    row = None
    for i in range(t.dim() - 2, -1, -1):  # axes of one element have no stride to speak of
        if t.shape[i] > 1:
            if row is not None and t.stride(i) != span:
                raise ValueError(f"{name}: row views need evenly spaced rows")
            if row is None:
                row = t.stride(i)
            span = t.stride(i) * t.shape[i]
    return t.shape[-1] if row is None else row


def ssd_norm_gate(y, z, weight, *, ngroups, eps=1e-5, out=None, stream=None):
    """out = weight * RMSNorm over `ngroups` groups of y * silu(z) (the norm first, then the gate);
    y [..., dim] contiguous, z [..., dim] may be a column slice of wider rows."""
    dev, dim = y.get_device(), y.shape[-1] if y.dim() else 0
    _need("y", y, y.shape, y.dtype, dev)
    _need("weight", weight, (dim,), torch.float32, dev)
    _need("out", out, y.shape, y.dtype, dev)
    zs = _rows_view("z", z, y, dev)
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty_like(y)
        _check(lib().ssd_norm_gate(y.numel() // dim if dim else 0, dim, ngroups, _dtype_code(y), _at(y), _at(z), zs,
                                   _at(weight), float(eps), _at(out), st), "ssd_norm_gate")
    return out


def _gate_norm_bwd(fn, y, z, weight, dout, ngroups, eps, want_dw, out, workspace, stream):
    dev, dim = y.get_device(), y.shape[-1] if y.dim() else 0
    _need("y", y, y.shape, y.dtype, dev)
    _need("weight", weight, (dim,), torch.float32, dev)
    _need("dout", dout, y.shape, y.dtype, dev)
    zs = _rows_view("z", z, y, dev)
    rows = y.numel() // dim if dim else 0
    o = dict(out or {})
    _need("dy", o.get("dy"), y.shape, y.dtype, dev)
    _need("dw", o.get("dw"), (dim,), torch.float32, dev)
    with _On(dev, stream) as st:
        if o.get("dy") is None:
            o["dy"] = torch.empty_like(y)
        if o.get("dz") is None:
            o["dz"] = torch.empty_like(y)
        if o.get("dw") is None:
            o["dw"] = torch.empty(dim, dtype=torch.float32, device=dev) if want_dw else None
        dzs = _rows_view("dz", o["dz"], y, dev)
        ws = _workspace(workspace, norm_bwd_workspace_bytes(rows, dim) if o["dw"] is not None else 0, dev)
        _check(getattr(lib(), fn)(rows, dim, ngroups, _dtype_code(y), _at(y), _at(z), zs, _at(weight), float(eps),
                                  _at(dout), _at(o["dy"]), _at(o["dz"]), dzs, _at(o["dw"]), _at(ws), _bytes(ws), st), fn)
    return o


def ssd_norm_gate_bwd(y, z, weight, dout, *, ngroups, eps=1e-5, want_dw: bool = True, out=None, workspace=None, stream=None):
    """Gradients of ssd_norm_gate: a dict dy, dz, dw (None unless want_dw); `out` may supply any of
    those tensors (dz may be a column slice of wider rows)."""
    return _gate_norm_bwd("ssd_norm_gate_bwd", y, z, weight, dout, ngroups, eps, want_dw, out, workspace, stream)


def ssd_gated_rmsnorm_bwd(y, z, weight, dout, *, ngroups, eps=1e-5, want_dw: bool = True, out=None, workspace=None,
                          stream=None):
    """Gradients of ssd_gated_rmsnorm, as ssd_norm_gate_bwd."""
    return _gate_norm_bwd("ssd_gated_rmsnorm_bwd", y, z, weight, dout, ngroups, eps, want_dw, out, workspace, stream)
