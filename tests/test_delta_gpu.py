"""GPU parity of the gated delta rule against the fp64 oracle on the same rounded inputs.

Tolerances, on ||got - ref|| / ||ref||, derived before any run from the unit roundings u (half a
step: bf16 2^-8, fp32 2^-24):
  fp32 storage        2e-5: dot products of up to 256 terms, 256 u = 1.5e-5 at worst, and the chain of
                      tokens does not grow it (unit keys and beta <= 1 make the state update a contraction)
  bf16, fp32 outputs  2e-5: the same, the inputs are exact (the tensor-core path keeps what enters the
                      state as two bf16 parts, 2^-16 of it lost at worst)
  bf16 outputs        3 * 2^-8: the output's own rounding, and at most two more in the products behind it
"""
import numpy as np
import pytest
import torch

import oracle
from ssd_cases import to_np
from state_space_sequence_chunked_b200 import _binding as ssd
from state_space_sequence_chunked_b200.inputs import Tensor

pytestmark = pytest.mark.gpu

F32_TOL, BF16_TOL = 2e-5, 3 * 2.0 ** -8


def draw(B, L, H, P, G, N, dtype, seed=0, h0=True, decay=1.0):
    r = np.random.default_rng(seed)
    k, q = r.standard_normal((B, L, G, N)), r.standard_normal((B, L, G, N))
    unit = lambda v: v / np.maximum(np.linalg.norm(v, axis=-1, keepdims=True), 1e-30)  # noqa: E731
    d = dict(x=r.standard_normal((B, L, H, P)), g=-decay * np.exp(r.uniform(np.log(1e-3), np.log(2.0), (B, L, H))),
             beta=1 / (1 + np.exp(-r.standard_normal((B, L, H)))), Bm=unit(k), Cm=unit(q))
    d = {n: Tensor(v, dtype) for n, v in d.items()}
    d["h0"] = Tensor(r.standard_normal((B, H, P, N)), "f32") if h0 else None
    d["dy"] = Tensor(r.standard_normal((B, L, H, P)), dtype)
    d["dh"] = Tensor(r.standard_normal((B, H, P, N)), "f32") if h0 else None
    return d


def on(d, device, names=("x", "g", "beta", "Bm", "Cm", "h0")):
    return [None if d[n] is None else d[n].torch(device) for n in names]


def ref_args(d):
    return [None if d[n] is None else d[n].value for n in ("x", "g", "beta", "Bm", "Cm", "h0")]


def err(got, ref):
    got = to_np(got)
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got))
    return float(np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30))


def tol(t, dtype):
    return BF16_TOL if t.dtype == torch.bfloat16 else F32_TOL


def check_fwd(d, device, dtype):
    a = on(d, device)
    y = torch.full_like(a[0], float("nan"))
    y, h = ssd.ssd_delta_fwd(*a, y=y)
    torch.cuda.synchronize()
    yr, hr = oracle.delta_recurrent(*ref_args(d))
    assert err(h, hr) <= F32_TOL
    assert err(y, yr) <= tol(y, dtype)


SHAPES = [  # B, L, H, P, G, N
    (1, 1, 1, 1, 1, 1), (2, 1, 4, 64, 2, 128), (1, 2, 3, 17, 3, 5), (2, 33, 4, 40, 2, 36), (1, 63, 2, 64, 1, 64),
    (1, 64, 2, 64, 2, 128), (2, 65, 4, 128, 2, 128), (1, 127, 3, 64, 1, 128), (3, 130, 6, 64, 2, 64), (1, 200, 2, 256, 1, 256),
    (1, 300, 2, 48, 1, 128), (1, 150, 5, 128, 5, 64), (1, 97, 2, 16, 1, 128), (2, 70, 2, 200, 2, 130), (1, 257, 2, 80, 2, 64),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(cuda_device, dtype, shape):
    check_fwd(draw(*shape, dtype, seed=sum(shape)), cuda_device, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_long_without_state(cuda_device, dtype):
    d = draw(1, 1500, 2, 64, 1, 128, dtype, seed=5, h0=False)
    check_fwd(d, cuda_device, dtype)
    y, h = ssd.ssd_delta_fwd(*on(d, cuda_device), return_final_state=False)
    y2, _ = ssd.ssd_delta_fwd(*on(d, cuda_device))
    torch.cuda.synchronize()
    assert h is None and torch.equal(y.view(torch.uint8), y2.view(torch.uint8))


EDGES = {
    "no decay": lambda d: d["g"].fill_(0.0),
    "strong decay": lambda d: d["g"].fill_(-60.0),
    "state cleared at tokens": lambda d: d["g"][:, [0, 3, 64, 70]].fill_(float("-inf")),
    "lowest value as a mask": lambda d: d["g"][:, [5, 63, 64]].fill_(torch.finfo(d["g"].dtype).min),
    "nothing written": lambda d: d["beta"].fill_(0.0),
    "all written": lambda d: d["beta"].fill_(1.0),
    "padded rows": lambda d: (d["beta"][:, 40:].zero_(), d["g"][:, 40:].zero_(), d["x"][:, 40:].fill_(7.0)),
    "one key throughout": lambda d: d["Bm"].copy_(d["Bm"][:, :1].expand_as(d["Bm"]).clone()),
    "zero keys": lambda d: d["Bm"][:, 10:90].zero_(),
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("edge", list(EDGES))
def test_edges_forward_and_backward(cuda_device, dtype, edge):
    """Every operator value stays finite where the recurrence is, and right."""
    d = draw(2, 135, 4, 64, 2, 128, dtype, seed=9)
    t = {n: v.torch(cuda_device).clone() for n, v in d.items()}
    EDGES[edge](t)
    args = [t[n] for n in ("x", "g", "beta", "Bm", "Cm", "h0")]
    refs = [to_np(v) for v in args]
    y, h = ssd.ssd_delta_fwd(*args)
    o = ssd.ssd_delta_bwd(*args, t["dy"], t["dh"])
    torch.cuda.synchronize()
    yr, hr = oracle.delta_recurrent(*refs)
    gr = oracle.delta_backward(*refs, to_np(t["dy"]), to_np(t["dh"]))
    assert err(h, hr) <= F32_TOL
    assert err(y, yr) <= tol(y, dtype)
    for n, ref in gr.items():
        if not np.any(ref):  # nothing written: no gradient through the write
            assert not torch.any(o[n]), n
        elif n == "dg" and edge in ("state cleared at tokens", "strong decay", "lowest value as a mask"):
            # a sum over the tokens of a chunk whose terms cancel where the decay leaves nothing: held
            # against the size of the terms, which dx (unit keys, unit state) measures
            got = to_np(o[n])
            assert np.all(np.isfinite(got))
            scale = np.linalg.norm(gr["dbeta"])
            assert np.linalg.norm(got - ref) <= tol(o[n], dtype) * max(scale, np.linalg.norm(ref)), n
        else:
            assert err(o[n], ref) <= tol(o[n], dtype), n


def check_bwd(d, device, dtype):
    a = on(d, device)
    dy, dh = on(d, device, ("dy", "dh"))
    o = ssd.ssd_delta_bwd(*a, dy, dh)
    torch.cuda.synchronize()
    ref = oracle.delta_backward(*ref_args(d), d["dy"].value, None if d["dh"] is None else d["dh"].value)
    for n, r in ref.items():
        assert err(o[n], r) <= tol(o[n], dtype), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(cuda_device, dtype, shape):
    check_bwd(draw(*shape, dtype, seed=1 + sum(shape)), cuda_device, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_many_heads_of_one_group(cuda_device, dtype):
    check_bwd(draw(1, 140, 12, 64, 1, 128, dtype, seed=21), cuda_device, dtype)
    check_bwd(draw(1, 140, 4, 64, 1, 128, dtype, seed=22, h0=False), cuda_device, dtype)


def test_gradients_by_differences(cuda_device):
    """The gradient kernels against differences of the forward kernel itself, fp32, along random
    directions: the forward's rounding over the step, 1e-6 / 2e-2, and the step's square."""
    d = draw(1, 70, 2, 64, 1, 64, "f32", seed=31)
    a = on(d, cuda_device)
    dy, dh = on(d, cuda_device, ("dy", "dh"))
    o = ssd.ssd_delta_bwd(*a, dy, dh)
    r = torch.Generator(device=cuda_device).manual_seed(1)
    for i, n in enumerate(("dx", "dg", "dbeta", "dB", "dC", "dh0")):
        v = torch.randn(a[i].shape, generator=r, device=cuda_device)
        v *= a[i].norm() / v.norm()
        ends = []
        for s in (1e-2, -1e-2):
            b = list(a)
            b[i] = a[i] + s * v
            y, h = ssd.ssd_delta_fwd(*b)
            ends.append(float((y.double() * dy).sum() + (h.double() * dh).sum()))
        want, got = (ends[0] - ends[1]) / 2e-2, float((o[n].double() * v).sum())
        size = float(o[n].double().norm() * v.double().norm()) / np.sqrt(v.numel())
        assert abs(want - got) <= 1e-2 * max(abs(got), size), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 4), (3, 4, 64, 2, 128), (2, 6, 33, 3, 36), (2, 2, 256, 1, 256), (65, 2, 8, 2, 132)],
                         ids=str)
@pytest.mark.parametrize("in_place", [True, False])
def test_step(cuda_device, dtype, shape, in_place):
    B, H, P, G, N = shape
    d = draw(B, 1, H, P, G, N, dtype, seed=sum(shape))
    x, g, beta, Bm, Cm, h0 = on(d, cuda_device)
    state = h0.clone()
    out = None if in_place else torch.full_like(h0, float("nan"))
    y = ssd.ssd_delta_decode_step(state, x[:, 0].clone(), g[:, 0].clone(), beta[:, 0].clone(), Bm[:, 0].clone(),
                                  Cm[:, 0].clone(), state_out=out)
    torch.cuda.synchronize()
    yr, hr = oracle.delta_recurrent(*ref_args(d))
    assert err(y, yr[:, 0]) <= tol(y, dtype)
    assert err(state if in_place else out, hr) <= F32_TOL
    if not in_place:
        assert torch.equal(state, h0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_then_steps_equal_one_pass(cuda_device, dtype):
    """Serving: a prefill in two pieces, then single tokens, against the whole sequence at once."""
    d = draw(2, 150, 4, 64, 2, 128, dtype, seed=41)
    a = on(d, cuda_device)
    cut = lambda lo, hi: [v[:, lo:hi].clone() for v in a[:5]]  # noqa: E731
    y1, h = ssd.ssd_delta_fwd(*cut(0, 100), a[5])
    y2, h = ssd.ssd_delta_fwd(*cut(100, 137), h)
    ys = [y1, y2]
    for t in range(137, 150):
        ys.append(ssd.ssd_delta_decode_step(h, *[v[:, t].clone() for v in a[:5]]).unsqueeze(1))
    torch.cuda.synchronize()
    yr, hr = oracle.delta_recurrent(*ref_args(d))
    assert err(torch.cat(ys, 1), yr) <= tol(y1, dtype)
    assert err(h, hr) <= F32_TOL


def test_empty_sequences(cuda_device):
    d = draw(2, 3, 4, 64, 2, 128, "bf16", seed=51)
    x, g, beta, Bm, Cm, h0 = on(d, cuda_device)
    none = [v[:, :0].contiguous() for v in (x, g, beta, Bm, Cm)]
    y, h = ssd.ssd_delta_fwd(*none, h0)
    _, z = ssd.ssd_delta_fwd(*none)
    o = ssd.ssd_delta_bwd(*none, h0, y, h0)
    o2 = ssd.ssd_delta_bwd(*none, None, y)
    nobody = [v[:0].contiguous() for v in (x, g, beta, Bm, Cm, h0)]
    yb, hb = ssd.ssd_delta_fwd(*nobody)
    torch.cuda.synchronize()
    assert torch.equal(h, h0) and not torch.any(z) and torch.equal(o["dh0"], h0) and not torch.any(o2["dh0"])
    assert yb.shape[0] == 0 and hb.shape[0] == 0


def test_neighbours_are_left_alone(cuda_device):
    """Outputs and workspace inside larger buffers: nothing is written outside them."""
    for shape in ((1, 67, 3, 40, 1, 36), (1, 67, 2, 64, 1, 128), (2, 65, 4, 128, 2, 128)):
        for dtype in ("f32", "bf16"):
            d = draw(*shape, dtype, seed=61)
            a = on(d, cuda_device)
            dy, dh = on(d, cuda_device, ("dy", "dh"))
            B, L, H, P, G, N = shape
            code = ssd.SSD_BF16 if dtype == "bf16" else ssd.SSD_F32
            bufs = []

            def inside(like_shape, dt):
                n = int(np.prod(like_shape))
                es = torch.empty(0, dtype=dt).element_size()
                pad = 256 // es
                buf = torch.full((n + 2 * pad,), 3.0, dtype=dt, device=cuda_device)
                bufs.append((buf, pad, n))
                return buf[pad:pad + n].view(like_shape)

            def ws(plan):
                n = plan["workspace_bytes"]
                buf = torch.full((n + 512,), 3, dtype=torch.uint8, device=cuda_device)
                bufs.append((buf, 256, n))
                return buf[256:256 + n]

            dt = a[0].dtype
            y, h = inside((B, L, H, P), dt), inside((B, H, P, N), torch.float32)
            ssd.ssd_delta_fwd(*a, y=y, h_final=h, workspace=ws(ssd.delta_fwd_plan(*shape, code)))
            out = {"dx": inside((B, L, H, P), dt), "dg": inside((B, L, H), dt), "dbeta": inside((B, L, H), dt),
                   "dB": inside((B, L, G, N), dt), "dC": inside((B, L, G, N), dt), "dh0": inside((B, H, P, N), torch.float32)}
            ssd.ssd_delta_bwd(*a, dy, dh, out=out, workspace=ws(ssd.delta_bwd_plan(*shape, code)))
            torch.cuda.synchronize()
            for buf, pad, n in bufs:
                assert bool((buf[:pad] == 3).all()) and bool((buf[pad + n:] == 3).all())


@pytest.mark.parametrize("shape", [(2, 200, 4, 64, 2, 128), (1, 70, 2, 40, 1, 36)], ids=str)
def test_graphs_streams_and_repeats(cuda_device, shape):
    """The same call on another stream, captured and replayed, on new inputs in the same buffers, and
    twice: the same bits each time."""
    d, e = draw(*shape, "bf16", seed=71), draw(*shape, "bf16", seed=72)
    names = ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh")
    a, b = on(d, cuda_device, names), on(e, cuda_device, names)

    def both(v, stream=None):
        y, h = ssd.ssd_delta_fwd(*v[:6], stream=stream)
        return [y, h] + list(ssd.ssd_delta_bwd(*v, stream=stream).values())

    same = lambda u, v: all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(u, v))  # noqa: E731
    want_a, want_b = both(a), both(b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(a, stream=s)
    s.synchronize()
    assert same(got, want_a)
    buf = [v.clone() for v in a]
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = both(buf)
    with torch.cuda.graph(graph2, pool=graph.pool()):
        two = both(buf)
    graph.replay()
    torch.cuda.synchronize()
    assert same(one, want_a)
    for t, v in zip(buf, b):
        t.copy_(v)
    graph2.replay()
    torch.cuda.synchronize()
    assert same(two, want_b)
    assert same(both(a), want_a)


def test_two_streams_at_once(cuda_device):
    d = [draw(2, 300, 4, 64, 2, 128, "bf16", seed=81 + i) for i in range(2)]
    a = [on(v, cuda_device, ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh")) for v in d]
    want = [list(ssd.ssd_delta_bwd(*v).values()) for v in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in a]
    got = [[list(ssd.ssd_delta_bwd(*v, stream=s).values()) for v, s in zip(a, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for round_ in got:
        for g, w in zip(round_, want):
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(g, w))


CUT = [(2, 130, 160, 16, 1, 64), (1, 200, 152, 72, 2, 64), (3, 100, 50, 136, 5, 128), (5, 330, 60, 64, 1, 128)]


@pytest.mark.parametrize("shape", CUT, ids=str)
def test_more_streams_than_sms(cuda_device, shape):
    """More head pairs (or heads) than SMs: streams are cut between CTAs and their state handed on."""
    d = draw(*shape, "bf16", seed=91)
    check_fwd(d, cuda_device, "bf16")
    check_bwd(d, cuda_device, "bf16")


def test_waits_that_run_out(cuda_device):
    """With a limit of 1 us some wait between the warps runs out: the call comes back, says so, and the
    next one at the normal limit is right."""
    shape = CUT[0]
    d = draw(*shape, "bf16", seed=92)
    a = on(d, cuda_device)
    n = ssd.delta_fwd_plan(*shape, ssd.SSD_BF16)["workspace_bytes"]
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_device)
    ssd.ssd_delta_fwd(*a, workspace=ws)
    assert ssd.delta_status(shape, ssd.SSD_BF16, ws) == 0
    try:
        ssd.set_wait_limit_us(1)
        ssd.ssd_delta_fwd(*a, workspace=ws)
        assert ssd.delta_status(shape, ssd.SSD_BF16, ws) == 6  # SSD_ERR_TIMEOUT
    finally:
        ssd.set_wait_limit_us(0)
    check_fwd(d, cuda_device, "bf16")
    assert ssd.delta_status((1, 4, 2, 64, 1, 64), ssd.SSD_BF16, None) == 0  # a path without waits
