"""Both paths of the gated delta rule where their own blocking shows: tiles of the tensor-core path that the sizes
do not fill, blocks of four tokens of the sequential one, lengths on both sides of the rule between them, streams
cut between CTAs inside graphs. Tolerances are those of test_delta_gpu.py.
"""
import numpy as np
import pytest
import torch

import oracle
from ssd_cases import to_np
from state_space_sequence_chunked_b200 import _binding as ssd
from test_delta_gpu import CUT, F32_TOL, check_bwd, check_fwd, draw, err, on, ref_args, tol

pytestmark = pytest.mark.gpu

PART = [  # B, L, H, P, G, N on the tensor cores, dstate and headdim away from whole tiles
    (1, 128, 2, 8, 1, 8), (2, 129, 3, 24, 1, 24), (1, 191, 4, 72, 2, 40), (1, 193, 2, 136, 1, 72), (2, 140, 6, 64, 3, 104),
    (1, 256, 7, 40, 1, 120), (1, 131, 3, 248, 1, 16), (4, 150, 25, 16, 1, 128),
]


@pytest.mark.parametrize("shape", PART, ids=str)
def test_part_filled_tiles(cuda_device, shape):
    assert ssd.delta_fwd_plan(*shape, ssd.SSD_BF16)["path"] == "tcgen05"
    d = draw(*shape, "bf16", seed=101)
    check_fwd(d, cuda_device, "bf16")
    check_bwd(d, cuda_device, "bf16")


ODD = [(1, 300, 3, 17, 1, 5), (2, 260, 4, 243, 2, 34), (1, 256, 2, 1, 1, 1), (1, 270, 6, 64, 3, 127), (3, 333, 2, 63, 1, 64)]


@pytest.mark.parametrize("h0", [True, False])
@pytest.mark.parametrize("shape", ODD, ids=str)
def test_sizes_of_no_whole_vectors(cuda_device, shape, h0):
    """On padded copies (from 8 on; smaller sizes in fp32); outputs stay within their own bounds and the call can
    be captured."""
    assert ssd.delta_fwd_plan(*shape, ssd.SSD_BF16)["path"] == ("tcgen05" if min(shape[3], shape[5]) >= 8 else "simt")
    d = draw(*shape, "bf16", seed=102, h0=h0)
    check_fwd(d, cuda_device, "bf16")
    check_bwd(d, cuda_device, "bf16")
    a = on(d, cuda_device)
    y, h = ssd.ssd_delta_fwd(*a)
    pad = torch.full((y.numel() + 64,), 3.0, dtype=y.dtype, device=cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.ssd_delta_fwd(*a, y=pad[32:32 + y.numel()].view(y.shape), return_final_state=False)
    graph.replay()
    torch.cuda.synchronize()
    assert same([pad[32:32 + y.numel()].view(y.shape)], [y])
    assert bool((pad[:32] == 3).all()) and bool((pad[32 + y.numel():] == 3).all())


@pytest.mark.parametrize("L", [1, 2, 3, 9, 31, 63])
@pytest.mark.parametrize("size", [(2, 5, 64, 1, 64), (1, 4, 16, 2, 128), (1, 3, 19, 1, 35)], ids=str)
def test_short_backward_on_tensor_cores(cuda_device, L, size):
    B, H, P, G, N = size
    assert ssd.delta_bwd_plan(B, L, H, P, G, N, ssd.SSD_BF16)["path"] == "tcgen05"
    check_bwd(draw(B, L, H, P, G, N, "bf16", seed=L), cuda_device, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [3, 33, 100, 129, 256])
@pytest.mark.parametrize("L", [1, 3, 4, 5, 8, 9, 17, 33, 34])
def test_blocks_of_four_tokens(cuda_device, dtype, N, L):
    d = draw(2, L, 3, 19, 1, N, dtype, seed=L + N)
    check_fwd(d, cuda_device, dtype)
    check_bwd(d, cuda_device, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", range(6))
def test_state_cleared_at_each_place_of_a_block(cuda_device, dtype, at):
    """A decay of minus infinity: what comes after does not see the state before."""
    d = draw(1, 11, 2, 16, 1, 36, dtype, seed=3)
    a = on(d, cuda_device)
    a[1] = a[1].clone()
    a[1][:, at] = float("-inf")
    y, h = ssd.ssd_delta_fwd(*a)
    torch.cuda.synchronize()
    yr, hr = oracle.delta_recurrent(*[to_np(v) for v in a])
    assert err(h, hr) <= F32_TOL and err(y, yr) <= tol(y, dtype)


@pytest.mark.parametrize("dtype,shape", [("f32", (1, 41, 2, 20, 1, 36)), ("bf16", (1, 41, 2, 20, 1, 36)),
                                         ("bf16", (2, 150, 4, 64, 2, 128))], ids=str)
@pytest.mark.parametrize("with_h0,with_dh,want", [(True, False, True), (False, True, True), (False, False, True), (True, True, False)])
def test_states_given_or_not(cuda_device, dtype, shape, with_h0, with_dh, want):
    d = draw(*shape, dtype, seed=7)
    a = on(d, cuda_device, ("x", "g", "beta", "Bm", "Cm"))
    h0, dy, dh = on(d, cuda_device, ("h0", "dy", "dh"))
    o = ssd.ssd_delta_bwd(*a, h0 if with_h0 else None, dy, dh if with_dh else None, want_dh0=want)
    torch.cuda.synchronize()
    ref = oracle.delta_backward(*ref_args(d)[:5], d["h0"].value if with_h0 else None, d["dy"].value, d["dh"].value if with_dh else None)
    assert (o["dh0"] is not None) == want
    for n, r in ref.items():
        if o[n] is not None:
            assert err(o[n], r) <= tol(o[n], dtype), n


@pytest.mark.parametrize("heads", [(1, 24), (8, 24), (32, 16)], ids=str)
@pytest.mark.parametrize("L", [2, 7, 20, 40, 127, 128])
def test_both_sides_of_the_path_rule(cuda_device, heads, L):
    B, H = heads
    check_fwd(draw(B, L, H, 64, 1, 128, "bf16", seed=L), cuda_device, "bf16")


def same(u, v):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(u, v))


@pytest.mark.parametrize("shape", CUT[:3], ids=str)
def test_cut_streams_in_graphs_and_on_two_streams(cuda_device, shape):
    d = [draw(*shape, "bf16", seed=111 + i) for i in range(2)]
    a = [on(v, cuda_device, ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh")) for v in d]

    def both(v, stream=None, ws=None):
        y, h = ssd.ssd_delta_fwd(*v[:6], stream=stream, workspace=ws)
        return [y, h] + list(ssd.ssd_delta_bwd(*v, stream=stream, workspace=ws).values())

    want = [both(v) for v in a]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in a]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[both(v, stream=s) for v, s in zip(a, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(same(g, w) for turn in got for g, w in zip(turn, want))
    # two graphs that share one workspace, replayed in turn
    need = max(p(*shape, ssd.SSD_BF16)["workspace_bytes"] for p in (ssd.delta_fwd_plan, ssd.delta_bwd_plan))
    ws = torch.empty(need, dtype=torch.uint8, device=cuda_device)
    graphs, outs = [], []
    for v in a:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(v, ws=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, want))


def test_status_after_a_backward_pass(cuda_device):
    """Of a length whose forward pass has no workspace and no waits, and whose backward pass has both."""
    shape = (1, 37, 4, 64, 1, 128)
    assert ssd.delta_fwd_plan(*shape, ssd.SSD_BF16)["workspace_bytes"] == 0
    d = draw(*shape, "bf16", seed=121)
    a = on(d, cuda_device, ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh"))
    ws = torch.empty(ssd.delta_bwd_plan(*shape, ssd.SSD_BF16)["workspace_bytes"], dtype=torch.uint8, device=cuda_device)
    ssd.ssd_delta_bwd(*a, workspace=ws)
    assert ssd.delta_status(shape, ssd.SSD_BF16, ws) == 0
    # What a kernel whose wait ran out leaves, set from the host: the waits of so short a call may all end
    # within the shortest limit, a microsecond.
    ws[0] = 1
    assert ssd.delta_status(shape, ssd.SSD_BF16, ws) == 6  # SSD_ERR_TIMEOUT
    ssd.ssd_delta_bwd(*a, workspace=ws)                    # the next call clears it
    assert ssd.delta_status(shape, ssd.SSD_BF16, ws) == 0
    check_bwd(d, cuda_device, "bf16")
    assert ssd.delta_status(shape, ssd.SSD_BF16, None) == 0


def test_many_slices_of_a_group(cuda_device):
    """One group of many heads over few chunks: the heads' gradients come in parts, also where they do not divide."""
    for H in (17, 48, 79):
        d = draw(1, 70, H, 8, 1, 40, "bf16", seed=H)
        assert ssd.delta_bwd_plan(1, 70, H, 8, 1, 40, ssd.SSD_BF16)["kernels"] == 4
        check_bwd(d, cuda_device, "bf16")


def test_values_that_are_not_numbers_stay_in_their_rows(cuda_device):
    """Infinite and NaN values of x in some state rows leave the other rows' outputs as they were."""
    for dtype, shape in (("f32", (1, 21, 2, 24, 1, 36)), ("bf16", (1, 200, 2, 64, 1, 128))):
        d = draw(*shape, dtype, seed=131)
        a = on(d, cuda_device)
        y, h = ssd.ssd_delta_fwd(*a)
        x = a[0].clone()
        x[:, 5, 0, 3] = float("inf")
        x[:, 9, 1, 7] = float("nan")
        y2, h2 = ssd.ssd_delta_fwd(x, *a[1:])
        torch.cuda.synchronize()
        for head, row in ((0, 3), (1, 7)):
            keep = [p for p in range(shape[3]) if p != row]
            assert same([y[:, :, head, keep].contiguous(), h[:, head, keep].contiguous()],
                        [y2[:, :, head, keep].contiguous(), h2[:, head, keep].contiguous()])
            assert not bool(torch.isfinite(h2[:, head, row]).all())


def test_orders_of_magnitude(cuda_device):
    """Strong decays right before and after a chunk's end, and values far from one."""
    d = draw(1, 260, 2, 64, 1, 128, "bf16", seed=141)
    a = on(d, cuda_device)
    a[1] = a[1].clone()
    a[1][:, [62, 63, 64, 65, 128, 191]] = -80.0
    a[0] = (a[0].float() * 1e4).bfloat16()
    a[5] = a[5] * 1e-3
    y, h = ssd.ssd_delta_fwd(*a)
    torch.cuda.synchronize()
    yr, hr = oracle.delta_recurrent(*[to_np(v) for v in a])
    assert err(h, hr) <= F32_TOL and err(y, yr) <= tol(y, "bf16")
    assert np.isfinite(yr).all()


BAD = {  # input, value at head 1 of four, token 20
    "NaN decay": ("g", float("nan")), "infinite decay": ("g", float("inf")), "NaN strength": ("beta", float("nan")),
    "infinite strength": ("beta", float("inf")), "an inverse that overflows": ("beta", 3e38), "infinite x": ("x", float("inf")),
    "NaN cotangent": ("dy", float("nan")),
}


@pytest.mark.parametrize("bad", list(BAD))
@pytest.mark.parametrize("dtype,shape", [("f32", (1, 41, 4, 24, 2, 36)), ("bf16", (1, 200, 4, 64, 2, 128)), ("bf16", (2, 150, 4, 40, 1, 64)),
                                         ("bf16", (1, 130, 4, 128, 2, 128))], ids=str)
def test_values_that_are_not_numbers_stay_in_their_head(cuda_device, dtype, shape, bad):
    """The definition keeps heads apart but for the gradients of shared keys and queries: one head's values that are not
    finite leave the others' outputs, states and own gradients as they were, bit by bit."""
    d = draw(*shape, dtype, seed=151)
    names = ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh")
    a = dict(zip(names, on(d, cuda_device, names)))
    if bad == "an inverse that overflows":
        a["Bm"][:, 20:30] = a["Bm"][:, 20:21].clone()  # keys alike: products of strengths in the inverse

    def run():
        y, h = ssd.ssd_delta_fwd(*[a[n] for n in names[:6]])
        o = ssd.ssd_delta_bwd(*[a[n] for n in names])
        torch.cuda.synchronize()
        return {"y": y, "h": h, "dx": o["dx"], "dg": o["dg"], "dbeta": o["dbeta"], "dh0": o["dh0"]}

    want = run()
    name, value = BAD[bad]
    if bad == "an inverse that overflows":
        a[name][:, 20:30, 1] = value
    else:
        a[name][:, 20, 1] = value
    got = run()
    axis = {"y": 2, "h": 1, "dx": 2, "dg": 2, "dbeta": 2, "dh0": 1}
    for n in want:
        for head in (0, 2, 3):
            assert torch.equal(got[n].select(axis[n], head), want[n].select(axis[n], head)), (n, head)
    assert not all(bool(torch.isfinite(got[n].select(axis[n], 1)).all()) for n in got)


@pytest.mark.parametrize("L", [1, 2, 3, 5, 17, 32, 33])
@pytest.mark.parametrize("size", [(2, 37, 128, 1, 64), (1, 48, 64, 2, 128), (1, 30, 40, 1, 24), (1, 21, 19, 1, 35)], ids=str)
def test_few_tokens_of_many_heads(cuda_device, L, size):
    """Gradients made of few numbers, that can be small against the heads' terms that cancel in them: without a state,
    one token's dB and dC are one number per batch row and group."""
    for seed in range(12 if L < 4 else 2):
        d = draw(size[0], L, *size[1:], "bf16", seed=1000 * L + seed, h0=seed % 3 == 0)
        check_bwd(d, cuda_device, "bf16")


@pytest.mark.parametrize("L", [1, 2, 4, 9, 20, 32])
@pytest.mark.parametrize("size", [(1, 1, 64, 1, 128), (1, 2, 128, 1, 64), (3, 1, 24, 1, 40), (1, 3, 35, 1, 19)], ids=str)
def test_few_tokens_of_few_heads(cuda_device, L, size):
    """dg and dbeta are few numbers as well."""
    for seed in range(10):
        check_bwd(draw(size[0], L, *size[1:], "bf16", seed=2000 * L + seed, h0=seed % 2 == 0), cuda_device, "bf16")
