"""GPU parity of the norms around a block, and of their gradients, against the fp64 oracle on the same
rounded inputs, and a gated-delta block run as a user runs it.

Tolerances on ||got - ref|| / ||ref||: fp32 outputs 2e-5 (row sums of at most 8192 terms in partial
sums, the fast exponential's 2^-21 and the square root), bf16 outputs 2^-8 (half a step) + 2e-5."""
import numpy as np
import pytest
import torch

import oracle
from ssd_cases import to_np
from state_space_sequence_chunked_b200 import _binding as ssd
from state_space_sequence_chunked_b200 import gated_delta
from state_space_sequence_chunked_b200.inputs import Tensor

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 2.0 ** -8 + 2e-5}
EPS = 1e-5


def close(got, ref, name=""):
    g = to_np(got)
    assert g.shape == ref.shape and np.all(np.isfinite(g)), name
    assert np.linalg.norm(g - ref) <= TOL[got.dtype] * max(np.linalg.norm(ref), 1e-30), name


def normal(r, shape, dtype, mean=0.0, sd=1.0):
    return Tensor(mean + sd * r.standard_normal(shape), dtype)


@pytest.mark.parametrize("dtype,rdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,dim", [(1, 1), (5, 33), (37, 64), (3, 130), (700, 128), (9, 2560), (4, 4098), (6, 8192), (1, 8191),
                                      (1300, 72)])
@pytest.mark.parametrize("parts", ["residual scale", "residual", "scale", ""])
def test_add_rmsnorm(cuda_device, dtype, rdtype, rows, dim, parts):
    r = np.random.default_rng(rows + dim)
    x, res = normal(r, (rows, dim), dtype), normal(r, (rows, dim), rdtype, sd=2.0) if "residual" in parts else None
    w, sc = normal(r, dim, "f32", 1.0, 0.1), normal(r, dim, "f32", 1.0, 0.3) if "scale" in parts else None
    t = lambda v: None if v is None else v.torch(cuda_device)  # noqa: E731
    v = lambda u: None if u is None else u.value  # noqa: E731
    out0 = torch.full((rows, dim), float("nan"), dtype=t(x).dtype, device=cuda_device)
    res0 = torch.full((rows, dim), float("nan"), dtype=torch.float32 if rdtype == "f32" else torch.bfloat16, device=cuda_device)
    got, out = ssd.ssd_add_rmsnorm(t(x), t(res), t(w), scale=t(sc), eps=EPS, res_out=res0, out=out0)
    want, out_ref = oracle.add_rmsnorm(x.value, v(res), w.value, scale=v(sc), eps=EPS)
    torch.cuda.synchronize()
    close(got, want, "r")
    close(out, out_ref, "out")
    # backward, from the sum as it was stored
    do, dr = normal(r, (rows, dim), dtype), normal(r, (rows, dim), rdtype) if "residual" in parts else None
    o = ssd.ssd_add_rmsnorm_bwd(got, t(w), t(do), t(dr), x=t(x), scale=t(sc), eps=EPS)
    ref = oracle.add_rmsnorm_backward(to_np(got), w.value, do.value, v(dr), x=x.value, scale=v(sc), eps=EPS)
    torch.cuda.synchronize()
    assert (o["dscale"] is None) == (sc is None)
    for n in ref:
        if n == "dres" or n == "dx" or n == "dw" or sc is not None:
            # dim = 1: out is the sign of r but for eps, and the gradient almost cancels
            if dim == 1 and n in ("dres", "dx", "dscale") and dr is None:
                off = TOL[o[n].dtype] * (np.linalg.norm(ref[n]) + 4 * np.linalg.norm(do.value))
                assert np.linalg.norm(to_np(o[n]) - ref[n]) <= off
            else:
                close(o[n], ref[n], n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,groups", [(1, 64, 1), (37, 512, 8), (5, 5120, 80), (650, 1536, 24), (3, 8192, 1), (7, 99, 3),
                                             (9, 66, 33), (4, 16384, 2), (2, 1000, 1), (11, 40, 40), (3, 257, 257)])
@pytest.mark.parametrize("zoff,zpad", [(0, 0), (8, 24), (2, 2), (1, 3)])
def test_gates(cuda_device, dtype, rows, dim, groups, zoff, zpad):
    """Both orders' gradients and the norm-first forward, z a column slice of wider rows at every
    alignment, dz written into the columns of wider rows."""
    r = np.random.default_rng(rows + dim + zoff)
    y, zw, do = normal(r, (rows, dim), dtype), normal(r, (rows, dim + zoff + zpad), dtype, sd=2.0), normal(r, (rows, dim), dtype)
    w = normal(r, dim, "f32", 1.0, 0.2)
    yt, wt, dot = (v.torch(cuda_device) for v in (y, w, do))
    zt = zw.torch(cuda_device)[:, zoff:zoff + dim]
    zv = zw.value[:, zoff:zoff + dim]
    out = ssd.ssd_norm_gate(yt, zt, wt, ngroups=groups, eps=EPS)
    torch.cuda.synchronize()
    close(out, oracle.norm_gate(y.value, zv, w.value, ngroups=groups, eps=EPS), "out")
    for fn, first in ((ssd.ssd_norm_gate_bwd, False), (ssd.ssd_gated_rmsnorm_bwd, True)):
        wide = torch.full_like(zw.torch(cuda_device), 5.0)
        o = fn(yt, zt, wt, dot, ngroups=groups, eps=EPS, out={"dz": wide[:, zoff:zoff + dim]})
        torch.cuda.synchronize()
        ref = oracle.gate_norm_backward(y.value, zv, w.value, do.value, ngroups=groups, eps=EPS, gate_first=first)
        for n in ref:
            if dim == groups and n in ("dy", "dz"):
                # groups of one channel a: their norm almost cancels the gradient, w do eps / (a^2 + eps)^1.5. What
                # is left where |a| is near sqrt(eps) is up to 300 times do, and the output's rounding is half a
                # step of that (the first term); the difference behind it has errors of the size of do (the second).
                off = TOL[o[n].dtype] * (np.linalg.norm(ref[n]) + 4 * np.linalg.norm(do.value))
                assert np.linalg.norm(to_np(o[n]) - ref[n]) <= off, n
            else:
                close(o[n], ref[n], n)
        assert bool((wide[:, :zoff] == 5).all()) and bool((wide[:, zoff + dim:] == 5).all())


def test_in_place(cuda_device):
    """The documented overlaps give the same bits as separate outputs."""
    r = torch.Generator(device=cuda_device).manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=r, device=cuda_device)  # noqa: E731
    x, res, w, sc = mk(50, 256).bfloat16(), mk(50, 256), mk(256), mk(256)
    want = ssd.ssd_add_rmsnorm(x, res, w, scale=sc)
    x2, res2 = x.clone(), res.clone()
    got = ssd.ssd_add_rmsnorm(x2, res2, w, scale=sc, res_out=res2, out=x2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    do, dr = mk(50, 256).bfloat16(), mk(50, 256)
    want = ssd.ssd_add_rmsnorm_bwd(res, w, do, dr, x=x, scale=sc)
    do2, dr2 = do.clone(), dr.clone()
    got = ssd.ssd_add_rmsnorm_bwd(res, w, do2, dr2, x=x, scale=sc, out={"dres": dr2, "dx": do2})
    assert all(torch.equal(got[n], want[n]) for n in want)
    y, z = mk(50, 256).bfloat16(), mk(50, 512).bfloat16()[:, 128:384]
    want_f = ssd.ssd_norm_gate(y, z, w, ngroups=4)
    for fn in (ssd.ssd_norm_gate_bwd, ssd.ssd_gated_rmsnorm_bwd):
        want = fn(y, z, w, do, ngroups=4)
        for target in ("y", "dout"):
            y2, do2 = y.clone(), do.clone()
            z2 = torch.empty(50, 512, dtype=torch.bfloat16, device=cuda_device)[:, 128:384]
            z2.copy_(z)
            got = fn(y2, z2, w, do2, ngroups=4, out={"dy": y2 if target == "y" else do2, "dz": z2})
            assert all(torch.equal(got[n], want[n]) for n in want)
    y2 = y.clone()
    assert torch.equal(ssd.ssd_norm_gate(y2, z, w, ngroups=4, out=y2), want_f)


def test_empty_rows(cuda_device):
    x, w = torch.empty(0, 64, device=cuda_device), torch.ones(64, device=cuda_device)
    res, out = ssd.ssd_add_rmsnorm(x, None, w)
    o = ssd.ssd_add_rmsnorm_bwd(x, w, x, out={"dw": torch.full((64,), 3.0, device=cuda_device)})
    p = ssd.ssd_norm_gate_bwd(x, x, w, x, ngroups=2, out={"dw": torch.full((64,), 3.0, device=cuda_device)})
    torch.cuda.synchronize()
    assert res.shape == out.shape == (0, 64) and not torch.any(o["dw"]) and not torch.any(p["dw"])


def test_captured_and_repeated(cuda_device):
    r = torch.Generator(device=cuda_device).manual_seed(5)
    mk = lambda *s: torch.randn(*s, generator=r, device=cuda_device)  # noqa: E731
    res, w, do = mk(3000, 640), mk(640), mk(3000, 640)

    def calls(stream=None):
        return [ssd.ssd_add_rmsnorm(do, res, w, stream=stream)[1],
                *[v for v in ssd.ssd_add_rmsnorm_bwd(res, w, do, x=do, scale=w, stream=stream).values()],
                *ssd.ssd_norm_gate_bwd(res, do, w, do, ngroups=5, stream=stream).values()]

    want = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    graph.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = calls(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(other, want))


def block_weights(r, cfg, device):
    t = lambda a, dt: Tensor(a, dt)  # noqa: E731
    HP, GN, H = cfg.d_inner, cfg.ngroups * cfg.dstate, cfg.nheads
    n = r.standard_normal
    w = dict(in_proj=t(n((cfg.d_in_proj, cfg.d_model)) / np.sqrt(cfg.d_model), "bf16"), conv_w=t(n((HP + 2 * GN, 4)) / 2, "f32"),
             conv_b=t(0.1 * n(HP + 2 * GN), "f32"), dt_bias=t(r.uniform(-5, -2, H), "f32"), A=t(-np.exp(r.uniform(0, 2, H)), "f32"),
             norm_w=t(1 + 0.1 * n(HP), "f32"), out_proj=t(n((cfg.d_model, HP)) / np.sqrt(HP), "bf16"))
    return w, gated_delta.DeltaWeights(**{k: v.torch(device) for k, v in w.items()})


def test_block_forward(cuda_device):
    """Two blocks on one residual stream against the oracle's composition in fp64. Each of the block's
    seven bf16 intermediates rounds once (2^-8 at worst, and the second block sees the first's)."""
    cfg = gated_delta.DeltaConfig(d_model=256, nheads=4, headdim=64, ngroups=2, dstate=128)
    r = np.random.default_rng(4)
    x = Tensor(r.standard_normal((2, 150, 256)), "bf16")
    pre = Tensor(1 + 0.1 * r.standard_normal(256), "f32")
    sc = Tensor(0.5 + 0.1 * r.standard_normal(256), "f32")
    w, wt = block_weights(r, cfg, cuda_device)
    v = {k: t.value for k, t in w.items()}

    def ref_block(u, res):
        res, n = oracle.add_rmsnorm(u, res, pre.value, scale=sc.value, eps=cfg.eps)
        row = n @ v["in_proj"].T
        HP, GN, H, N = cfg.d_inner, cfg.ngroups * cfg.dstate, cfg.nheads, cfg.dstate
        xs, Bm, Cm, dt = oracle.conv_split(row[..., HP:2 * HP + 2 * GN], row[..., 2 * HP + 2 * GN:2 * HP + 2 * GN + H], v["conv_w"],
                                           v["conv_b"], v["dt_bias"], nheads=H, headdim=cfg.headdim, ngroups=cfg.ngroups, dstate=N)
        unit = lambda t: t / np.sqrt(np.sum(t * t, axis=-1, keepdims=True) + cfg.key_eps)  # noqa: E731
        y, h = oracle.delta_recurrent(xs, dt * v["A"], 1 / (1 + np.exp(-row[..., 2 * HP + 2 * GN + H:])), unit(Bm),
                                      unit(Cm) / np.sqrt(N))
        o = oracle.norm_gate(y.reshape(*u.shape[:2], HP), row[..., :HP], v["norm_w"], ngroups=H, eps=cfg.eps)
        return o @ v["out_proj"].T, res, h

    res, res_ref, u, u_ref = None, None, x.torch(cuda_device), x.value
    for _ in range(2):
        u, res, h = gated_delta.block_fwd(u, res, wt, cfg, pre.torch(cuda_device), scale=sc.torch(cuda_device))
        u_ref, res_ref, h_ref = ref_block(u_ref, res_ref)
    torch.cuda.synchronize()
    for got, ref in ((u, u_ref), (res, res_ref), (h, h_ref)):
        got = to_np(got)
        assert np.all(np.isfinite(got))
        assert np.linalg.norm(got - ref) <= 14 * 2.0 ** -8 * np.linalg.norm(ref)


def test_block_core_gradients(cuda_device):
    """A training step's chain through the operators, forward and back by hand: the residual norm, unit
    keys, the delta rule, the gated norm, against fp64 adjoints chained the same way. fp32, so each
    link's bound is its own and five of them add."""
    B, L, H, P, G, N = 2, 90, 4, 32, 2, 64
    r = np.random.default_rng(14)
    d, n = H * P + 2 * G * N, r.standard_normal
    v = {k: Tensor(a, "f32").value for k, a in dict(
        x=n((B, L, d)), res=n((B, L, d)), pre=1 + 0.1 * n(d), g=-np.exp(n((B, L, H)) - 2), beta=1 / (1 + np.exp(-n((B, L, H)))),
        z=n((B, L, H * P)), w=1 + 0.1 * n(H * P), dout=n((B, L, H * P)), dres=n((B, L, d)), sc=1 + 0.1 * n(d)).items()}
    t = {k: torch.from_numpy(a).float().to(cuda_device) for k, a in v.items()}
    unit_v, key_eps = np.full(N, N ** -0.5), 1e-6
    unit = torch.from_numpy(unit_v).float().to(cuda_device)

    def split(a):
        xs, k, q = a[..., :H * P], a[..., H * P:H * P + G * N], a[..., H * P + G * N:]
        return xs.reshape(B, L, H, P), k.reshape(B, L, G, N), q.reshape(B, L, G, N)

    # forward
    res, a = ssd.ssd_add_rmsnorm(t["x"], t["res"], t["pre"], scale=t["sc"], eps=EPS)
    xs, k, q = (u.contiguous() for u in split(a))
    _, kn = ssd.ssd_add_rmsnorm(k, None, unit, eps=key_eps / N, want_res=False)
    _, qn = ssd.ssd_add_rmsnorm(q, None, unit, eps=key_eps / N, want_res=False)
    y, _ = ssd.ssd_delta_fwd(xs, t["g"], t["beta"], kn, qn)
    out = ssd.ssd_norm_gate(y.view(B, L, H * P), t["z"], t["w"], ngroups=H, eps=EPS)
    # and back
    go = ssd.ssd_norm_gate_bwd(y.view(B, L, H * P), t["z"], t["w"], t["dout"], ngroups=H, eps=EPS)
    gd = ssd.ssd_delta_bwd(xs, t["g"], t["beta"], kn, qn, None, go["dy"].view(B, L, H, P), want_dh0=False)
    gk = ssd.ssd_add_rmsnorm_bwd(k, unit, gd["dB"], eps=key_eps / N, want_dw=False)
    gq = ssd.ssd_add_rmsnorm_bwd(q, unit, gd["dC"], eps=key_eps / N, want_dw=False)
    da = torch.cat([gd["dx"].view(B, L, -1), gk["dx"].view(B, L, -1), gq["dx"].view(B, L, -1)], -1)
    ga = ssd.ssd_add_rmsnorm_bwd(res, t["pre"], da, t["dres"], x=t["x"], scale=t["sc"], eps=EPS)
    torch.cuda.synchronize()

    r_res, r_a = oracle.add_rmsnorm(v["x"], v["res"], v["pre"], scale=v["sc"], eps=EPS)
    r_xs, r_k, r_q = split(r_a)
    r_kn = oracle.add_rmsnorm(r_k, None, unit_v, eps=key_eps / N)[1]
    r_qn = oracle.add_rmsnorm(r_q, None, unit_v, eps=key_eps / N)[1]
    r_y, _ = oracle.delta_recurrent(r_xs, v["g"], v["beta"], r_kn, r_qn)
    r_y = r_y.reshape(B, L, H * P)
    r_out = oracle.norm_gate(r_y, v["z"], v["w"], ngroups=H, eps=EPS)
    r_go = oracle.gate_norm_backward(r_y, v["z"], v["w"], v["dout"], ngroups=H, eps=EPS, gate_first=False)
    r_gd = oracle.delta_backward(r_xs, v["g"], v["beta"], r_kn, r_qn, None, r_go["dy"].reshape(B, L, H, P))
    r_gk = oracle.add_rmsnorm_backward(r_k, unit_v, r_gd["dB"], eps=key_eps / N)["dx"]
    r_gq = oracle.add_rmsnorm_backward(r_q, unit_v, r_gd["dC"], eps=key_eps / N)["dx"]
    r_da = np.concatenate([r_gd["dx"].reshape(B, L, -1), r_gk.reshape(B, L, -1), r_gq.reshape(B, L, -1)], -1)
    r_ga = oracle.add_rmsnorm_backward(r_res, v["pre"], r_da, v["dres"], x=v["x"], scale=v["sc"], eps=EPS)
    pairs = [(out, r_out, "out")] + [(go[m], r_go[m], m) for m in ("dz", "dw")] + [(gd[m], r_gd[m], m) for m in ("dg", "dbeta")]
    pairs += [(ga[m], r_ga[m], m) for m in ("dres", "dx", "dw", "dscale")]
    for got, ref, name in pairs:
        assert np.linalg.norm(to_np(got) - ref) <= 5 * TOL[torch.float32] * np.linalg.norm(ref), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_of_negative_values(cuda_device, dtype):
    """Where the gate is small, against each value's own size. Half steps u = 2^-24: the exponential 4 u, the quotient 2 u,
    the square root 4 u, sums of 64 squares in eights and three exchanges 11 / 2 u, and a dozen products and sums: below
    32 u = 2^-19; the output's rounding to bf16 2^-8 more. dz of the norm-first order has the same factors."""
    r = np.random.default_rng(5)
    rows, dim, groups = 300, 512, 8
    y, do, w = normal(r, (rows, dim), dtype), normal(r, (rows, dim), dtype), normal(r, dim, "f32", 1.0, 0.1)
    z = Tensor(r.uniform(-80.0, -10.0, (rows, dim)), dtype)
    yt, zt, wt, dot = (v.torch(cuda_device) for v in (y, z, w, do))
    out = ssd.ssd_norm_gate(yt, zt, wt, ngroups=groups, eps=EPS)
    dz = ssd.ssd_norm_gate_bwd(yt, zt, wt, dot, ngroups=groups, eps=EPS)["dz"]
    torch.cuda.synchronize()
    off = 2.0 ** -19 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    ref = oracle.gate_norm_backward(y.value, z.value, w.value, do.value, ngroups=groups, eps=EPS, gate_first=False)["dz"]
    for got, want in ((out, oracle.norm_gate(y.value, z.value, w.value, ngroups=groups, eps=EPS)), (dz, ref)):
        assert np.all(np.abs(to_np(got) - want) <= off * np.abs(want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_at_its_ends(cuda_device, dtype):
    """Large and infinite z: the gate is z or 0, and a NaN stays in its channel."""
    z = torch.tensor([[100.0, 1e4, float("inf"), -100.0, -1e4, float("nan"), 0.0, 1.0]], device=cuda_device)
    y = torch.ones(1, 8, device=cuda_device)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    out = ssd.ssd_norm_gate(y.to(dt), z.to(dt), torch.ones(8, device=cuda_device), ngroups=1, eps=0.0).float()
    torch.cuda.synchronize()
    want = torch.tensor([100.0, 1e4, float("inf"), 0.0, 0.0, float("nan"), 0.0, 1 / (1 + np.exp(-1.0))], dtype=torch.float32,
                        device=cuda_device)
    assert torch.equal(torch.isnan(out[0]), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.allclose(out[0][fine], want[fine], rtol=2.0 ** -8 if dtype == "bf16" else 2.0 ** -19, atol=1e-30)
