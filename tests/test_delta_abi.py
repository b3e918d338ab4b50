"""The gated delta rule's and the norms' entry points without a GPU: plans and refusals, all before
anything is launched."""
import ctypes
import os
import re

import pytest
import torch

from state_space_sequence_chunked_b200 import _binding as B
from state_space_sequence_chunked_b200 import build as build_mod

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = range(5)
A16 = 4096  # a made-up aligned address: never dereferenced on the host
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def fwd(lib, shape=(2, 100, 4, 64, 2, 128), dtype=B.SSD_BF16, *, null=(), odd=(), ws=A16, ws_bytes=BIG):
    names = ("x", "g", "beta", "Bm", "Cm", "h0", "y", "h_final")
    p = [None if n in null else A16 + (4 if n in odd else 0) for n in names]
    return lib.ssd_delta_fwd(ctypes.byref(B.ShapeT(*shape)), dtype, *p, ws, ws_bytes, None)


def bwd(lib, shape=(2, 100, 4, 64, 2, 128), dtype=B.SSD_BF16, *, null=(), odd=(), ws=A16, ws_bytes=BIG):
    names = ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh_final", "dx", "dg", "dbeta", "dBm", "dCm", "dh0")
    p = [None if n in null else A16 + (4 if n in odd else 0) for n in names]
    return lib.ssd_delta_bwd(ctypes.byref(B.ShapeT(*shape)), dtype, *p, ws, ws_bytes, None)


def step(lib, shape=(2, 1, 4, 64, 2, 128), dtype=B.SSD_BF16, *, null=(), odd=(), state=1 << 30, state_out=1 << 40):
    names = ("state", "state_out", "x", "g", "beta", "Bm", "Cm", "y")
    at = dict(state=state, state_out=state_out)
    p = [None if n in null else at.get(n, A16) + (4 if n in odd else 0) for n in names]
    return lib.ssd_delta_decode_step(ctypes.byref(B.ShapeT(*shape)), dtype, *p, None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_shapes_and_types_are_checked(lib, call):
    L = 1 if call is step else 100
    assert call(lib, (0, L, 4, 64, 2, 128)) == OK  # nothing to do
    assert call(lib, (-1, L, 4, 64, 2, 128)) == INVALID
    assert call(lib, (2, -1, 4, 64, 2, 128)) == INVALID
    assert call(lib, (2, L, 4, 64, 3, 128)) == INVALID
    assert call(lib, (2, L, 0, 64, 1, 128)) == INVALID
    assert call(lib, (2, L, 4, 257, 2, 128)) == UNSUPPORTED
    assert call(lib, (2, L, 4, 64, 2, 260)) == UNSUPPORTED
    assert call(lib, (65536, L, 4, 64, 2, 128)) == UNSUPPORTED
    assert call(lib, dtype=7) == INVALID


@pytest.mark.parametrize("call,required", [(fwd, ("x", "g", "beta", "Bm", "Cm", "y")),
                                           (bwd, ("x", "g", "beta", "Bm", "Cm", "dy", "dx", "dg", "dbeta", "dBm", "dCm")),
                                           (step, ("state", "state_out", "x", "g", "beta", "Bm", "Cm", "y"))])
def test_pointers_are_checked(lib, call, required):
    for n in required:
        assert call(lib, null=(n,)) == INVALID, n
        assert call(lib, odd=(n,)) == ALIGNMENT, n
    for n in {fwd: ("h0", "h_final"), bwd: ("h0", "dh_final", "dh0"), step: ()}[call]:
        assert call(lib, odd=(n,)) == ALIGNMENT, n


def test_step_refusals(lib):
    assert step(lib, (2, 2, 4, 64, 2, 128)) == INVALID    # one token only
    assert step(lib, (2, 1, 4, 64, 2, 126)) == UNSUPPORTED
    size = 2 * 4 * 64 * 128 * 4
    assert step(lib, state_out=(1 << 30) + size - 16) == INVALID  # partly over the state
    assert step(lib, state_out=(1 << 30) - size + 16) == INVALID


@pytest.mark.parametrize("call,plan", [(fwd, B.delta_fwd_plan), (bwd, B.delta_bwd_plan)])
def test_workspace_is_checked(lib, call, plan):
    need = plan(2, 100, 4, 64, 2, 128, B.SSD_BF16)["workspace_bytes"]
    if need:
        assert call(lib, ws=None) == WORKSPACE
        assert call(lib, ws_bytes=need - 1) == WORKSPACE
    assert call(lib, odd=(), ws=A16 + 8) == ALIGNMENT


def test_plans(lib):
    for plan in (B.delta_fwd_plan, B.delta_bwd_plan):
        assert plan(2, 0, 4, 64, 2, 128, B.SSD_BF16) == {"path": "none", "kernels": 0, "workspace_bytes": 0}
        assert plan(0, 9, 4, 64, 2, 128, B.SSD_BF16)["path"] == "none"
        assert plan(1, 9, 4, 64, 2, 128, B.SSD_F32)["path"] == "simt"
        assert plan(1, 999, 4, 40, 2, 136, B.SSD_BF16)["path"] == "simt"
    for f in (lib.ssd_delta_fwd_plan, lib.ssd_delta_bwd_plan):
        assert f(ctypes.byref(B.ShapeT(1, 1, 1, 1, 1, 1)), 0, None) == INVALID


def add(lib, rows=4, dim=64, dtype=B.SSD_BF16, rdtype=B.SSD_F32, eps=1e-5, null=(), odd=()):
    p = {n: None if n in null else A16 + (4 if n in odd else 0) for n in ("x", "residual", "scale", "weight", "res_out", "out")}
    return lib.ssd_add_rmsnorm(rows, dim, dtype, rdtype, p["x"], p["residual"], p["scale"], p["weight"], eps, p["res_out"],
                               p["out"], None)


def add_bwd(lib, rows=4, dim=64, dtype=B.SSD_BF16, rdtype=B.SSD_F32, eps=1e-5, null=(), odd=(), ws=A16, ws_bytes=BIG):
    names = ("res", "weight", "dout", "dres_in", "x", "scale", "dres", "dx", "dw", "dscale")
    p = {n: None if n in null else A16 + (4 if n in odd else 0) for n in names}
    v = list(p.values())
    return lib.ssd_add_rmsnorm_bwd(rows, dim, dtype, rdtype, *v[:2], eps, *v[2:], ws, ws_bytes, None)


def gate(lib, rows=4, dim=64, groups=2, dtype=B.SSD_BF16, zs=64, eps=1e-5, null=(), odd=()):
    p = {n: None if n in null else A16 + (4 if n in odd else 0) for n in ("y", "z", "weight", "out")}
    return lib.ssd_norm_gate(rows, dim, groups, dtype, p["y"], p["z"], zs, p["weight"], eps, p["out"], None)


def gate_bwd(lib, rows=4, dim=64, groups=2, dtype=B.SSD_BF16, zs=64, eps=1e-5, null=(), odd=(), ws=A16, ws_bytes=BIG,
             first=False, dzs=64, z=A16, dz=1 << 30):
    names = ("y", "z", "weight", "dout", "dy", "dz", "dw")
    at = dict(z=z, dz=dz)
    p = {n: None if n in null else at.get(n, A16) + (4 if n in odd else 0) for n in names}
    f = lib.ssd_gated_rmsnorm_bwd if first else lib.ssd_norm_gate_bwd
    return f(rows, dim, groups, dtype, p["y"], p["z"], zs, p["weight"], eps, p["dout"], p["dy"], p["dz"], dzs, p["dw"], ws,
             ws_bytes, None)


@pytest.mark.parametrize("call", [add, gate, gate_bwd])
def test_norm_arguments(lib, call):
    big = {} if call is add else {"zs": 1 << 20} if call is gate else {"zs": 1 << 20, "dzs": 1 << 20}
    assert call(lib, rows=-1) == INVALID
    assert call(lib, dim=0) == INVALID
    assert call(lib, eps=-1.0) == INVALID
    assert call(lib, eps=float("nan")) == INVALID
    assert call(lib, dtype=3) == INVALID
    assert call(lib, dim=2 * 8200, **big) == UNSUPPORTED
    if call is not add:
        assert call(lib, groups=0) == INVALID
        assert call(lib, groups=3) == INVALID
        assert call(lib, zs=63) == INVALID
    if call is not gate_bwd:
        assert call(lib, rows=0) == OK


def test_add_norm_refusals(lib):
    assert add(lib, dtype=B.SSD_F32, rdtype=B.SSD_BF16) == UNSUPPORTED
    assert add(lib, rdtype=5) == INVALID
    for n in ("x", "weight", "out"):
        assert add(lib, null=(n,)) == INVALID, n
    for n in ("x", "residual", "scale", "weight", "res_out", "out"):
        assert add(lib, odd=(n,)) == ALIGNMENT, n
    for n in ("res", "weight", "dout"):
        assert add_bwd(lib, null=(n,)) == INVALID, n
    assert add_bwd(lib, null=("x",)) == INVALID          # dscale needs x
    for n in ("res", "weight", "dout", "dres_in", "x", "scale", "dres", "dx", "dw", "dscale"):
        assert add_bwd(lib, odd=(n,)) == ALIGNMENT, n
    assert add_bwd(lib, dtype=B.SSD_F32, rdtype=B.SSD_BF16) == UNSUPPORTED


def test_norm_bwd_workspace(lib):
    need = B.norm_bwd_workspace_bytes(4, 64)
    assert need > 0 and B.norm_bwd_workspace_bytes(0, 64) == 0
    for call in (add_bwd, gate_bwd):
        assert call(lib, ws=None) == WORKSPACE
        assert call(lib, ws_bytes=need - 1) == WORKSPACE
        assert call(lib, ws=A16 + 4) == ALIGNMENT
    assert lib.ssd_norm_bwd_workspace_bytes(-1, 64, ctypes.byref(ctypes.c_size_t())) == INVALID
    assert lib.ssd_norm_bwd_workspace_bytes(1, 64, None) == INVALID


@pytest.mark.parametrize("first", [False, True])
def test_gate_bwd_refusals(lib, first):
    for n in ("y", "z", "weight", "dout", "dy", "dz"):
        assert gate_bwd(lib, null=(n,), first=first) == INVALID, n
    for n in ("y", "weight", "dout", "dy", "dw"):
        assert gate_bwd(lib, odd=(n,), first=first) == ALIGNMENT, n
    assert gate_bwd(lib, z=A16 + 1, first=first) == ALIGNMENT
    assert gate_bwd(lib, dzs=63, first=first) == INVALID
    # dz over other rows of z, and over its columns at another offset
    assert gate_bwd(lib, z=1 << 20, dz=(1 << 20) + 128, first=first) == INVALID
    assert gate_bwd(lib, z=1 << 20, dz=(1 << 20) + 64, zs=128, dzs=128, first=first) == INVALID


def test_binding_refuses_wrong_tensors():
    """The binding's own checks need no GPU: they come before the call."""
    x = torch.zeros(1, 3, 2, 8)
    with pytest.raises(ValueError):
        B.ssd_delta_fwd(x, x[..., 0].contiguous(), x[..., 0].contiguous(), x, x)  # not on a GPU
    with pytest.raises(ValueError):
        B.ssd_delta_decode_step(x, x, x, x, x, x)
    with pytest.raises(ValueError):
        B.ssd_add_rmsnorm(x, None, torch.ones(8))
    with pytest.raises(ValueError):
        B.ssd_norm_gate(x, x, torch.ones(8), ngroups=1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int16, torch.int8, torch.uint8, torch.bool, torch.float8_e4m3fn])
def test_binding_refuses_types_of_the_residual_stream(dtype):
    """Types other than fp32 and bf16 are refused, also where the residual or res_out alone has them: read as bf16,
    a type of one byte would end before the kernel does."""
    other = torch.zeros(3, 8).to(dtype)
    for x in (torch.zeros(3, 8), torch.zeros(3, 8, dtype=torch.bfloat16)):
        w = torch.ones(8)
        for args in (dict(residual=other), dict(residual=None, res_out=other), dict(residual=other, res_out=other)):
            with pytest.raises(TypeError):
                B.ssd_add_rmsnorm(x, weight=w, **args)
        with pytest.raises(TypeError):
            B.ssd_add_rmsnorm_bwd(other, w, x)
    with pytest.raises(TypeError):
        B.ssd_add_rmsnorm(other, None, torch.ones(8))


def test_row_views():
    like = torch.zeros(3, 4, 8)
    wide = torch.zeros(3, 4, 20)
    cpu = like.get_device()
    assert B._rows_view("z", wide[..., 5:13], like, cpu) == 20
    assert B._rows_view("z", like, like, cpu) == 8
    assert B._rows_view("z", wide[:1, :1, :8], like[:1, :1], cpu) == 8
    assert B._rows_view("z", wide[:, :1, :8], like[:, :1], cpu) == 80
    with pytest.raises(ValueError):
        B._rows_view("z", torch.zeros(3, 8, 4).transpose(1, 2).contiguous().transpose(0, 1)[:3, :3], like, cpu)
    with pytest.raises(ValueError):
        B._rows_view("z", torch.zeros(3, 4, 16)[..., ::2], like, cpu)
    with pytest.raises(ValueError):  # rows of the first axis are not evenly spaced with the second's
        B._rows_view("z", torch.zeros(3, 6, 8)[:, :4], like, cpu)


def test_plan_rule(lib):
    """The forward's rule of length and heads, the backward's of sizes alone; sizes past the range are refused."""
    fwd_path = lambda *s: B.delta_fwd_plan(*s, B.SSD_BF16)["path"]  # noqa: E731
    assert fwd_path(1, 127, 24, 64, 1, 128) == "simt" and fwd_path(1, 128, 24, 64, 1, 128) == "tcgen05"
    assert fwd_path(8, 21, 24, 64, 1, 128) == "simt" and fwd_path(8, 22, 24, 64, 1, 128) == "tcgen05"
    assert fwd_path(32, 2, 80, 64, 1, 128) == "tcgen05"
    assert fwd_path(1, 255, 4, 40, 2, 36) == "simt" and fwd_path(1, 256, 4, 40, 2, 36) == "tcgen05"  # padded copies
    assert B.delta_fwd_plan(1, 256, 4, 40, 2, 36, B.SSD_BF16)["kernels"] == 4
    for L in (1, 37, 128):
        plan = B.delta_bwd_plan(1, L, 4, 64, 1, 128, B.SSD_BF16)
        assert plan["path"] == "tcgen05" and plan["workspace_bytes"] > 0
    for size in ((4, 264, 1, 16), (4, 16, 1, 264)):
        with pytest.raises(B.SSDError):
            B.delta_fwd_plan(1, 131, *size, B.SSD_BF16)


def test_grids_ask_the_device():
    """The launch rules of these kernels take the number of SMs from the device, not from a constant."""
    csrc = os.path.join(os.path.dirname(B.LIB_PATH), "csrc")
    for name in sorted(os.listdir(csrc)):
        if name.startswith(("ssd_delta", "ssd_norm", "delta_tc")):
            with open(os.path.join(csrc, name)) as f:
                code = re.sub(r"//[^\n]*", "", f.read())
            assert not re.search(r"\b14[78]\b", code), name
