"""The gradient of the log decay where the decay leaves little: dg shrinks like exp(g), and is held against its own
norm, against the fp64 oracle on the same rounded inputs.

Tolerances are those of test_delta_gpu.py: dg is a sum of products that all carry exp(g) of its token, so no term
cancels that is larger than the result. fp32 2e-5; bf16 3 * 2^-8 (its own rounding, and at most two more, of the
operands S, D, u and r, in each product).
"""
import pytest
import torch

import numpy as np
import oracle
from ssd_cases import to_np
from state_space_sequence_chunked_b200 import _binding as ssd
from test_delta_gpu import draw, err, on, tol

pytestmark = pytest.mark.gpu

SIZES = [  # general path, segments of 32; tensor cores, chunks of 64, in pairs, one head at a time, on padded copies
    ("f32", (1, 70, 2, 40, 1, 36)), ("f32", (2, 100, 4, 64, 2, 128)), ("bf16", (1, 75, 2, 24, 1, 136)),
    ("bf16", (1, 200, 4, 64, 2, 128)), ("bf16", (2, 135, 24, 64, 1, 64)), ("bf16", (1, 150, 2, 200, 1, 72)), ("bf16", (1, 131, 3, 43, 1, 34)),
]


def gradients(dtype, shape, change, device, seed):
    """(the kernels' gradients, the oracle's) with g changed in place."""
    d = draw(*shape, dtype, seed=seed)
    names = ("x", "g", "beta", "Bm", "Cm", "h0", "dy", "dh")
    a = dict(zip(names, (v.clone() for v in on(d, device, names))))
    change(a["g"])
    o = ssd.ssd_delta_bwd(*[a[n] for n in names])
    torch.cuda.synchronize()
    return o, oracle.delta_backward(*[to_np(a[n]) for n in names])


def index(t, at):
    return torch.tensor(at, device=t.device)


@pytest.mark.parametrize("g", [-0.5, -3.0, -5.0, -8.0, -12.0, -16.0, -30.0])
@pytest.mark.parametrize("dtype,shape", SIZES, ids=str)
def test_uniform_decay(cuda_device, dtype, shape, g):
    o, ref = gradients(dtype, shape, lambda t: t.fill_(g), cuda_device, seed=201)
    assert np.linalg.norm(ref["dg"]) > 0
    assert err(o["dg"], ref["dg"]) <= tol(o["dg"], dtype)


@pytest.mark.parametrize("dtype,shape", SIZES, ids=str)
def test_strong_decays_among_weak_ones(cuda_device, dtype, shape):
    """The gradients at the strongly decayed tokens alone, which the others' would hide."""
    at = [1, 2, 15, 16, 31, 32, 47, 48, 62, 63, 64, 69]
    o, ref = gradients(dtype, shape, lambda t: t.index_fill_(1, index(t, at), -14.0), cuda_device, seed=202)
    assert err(o["dg"][:, at], ref["dg"][:, at]) <= tol(o["dg"], dtype)
    assert err(o["dg"], ref["dg"]) <= tol(o["dg"], dtype)


@pytest.mark.parametrize("dtype,shape", SIZES, ids=str)
@pytest.mark.parametrize("value", [float("-inf"), -1e30])
def test_nothing_passes_a_cleared_state(cuda_device, dtype, shape, value):
    at = [0, 3, 15, 16, 31, 32, 63, 64]
    o, ref = gradients(dtype, shape, lambda t: t.index_fill_(1, index(t, at), value), cuda_device, seed=203)
    for n, r in ref.items():
        assert err(o[n], r) <= tol(o[n], dtype), n
    assert not np.any(ref["dg"][:, at]) and not bool(torch.any(o["dg"][:, at]))


@pytest.mark.parametrize("dtype,shape", SIZES, ids=str)
@pytest.mark.parametrize("value", [float("-inf"), -1e30])
def test_forward_of_a_cleared_state(cuda_device, dtype, shape, value):
    """Sequences of the general path's length and, on tensor cores, of whole and cut chunks."""
    for L in (shape[1], 300):
        d = draw(shape[0], L, *shape[2:], dtype, seed=204)
        a = [v.clone() for v in on(d, cuda_device)]
        a[1].index_fill_(1, index(a[1], [0, 3, 15, 16, 31, 32, 63, 64]), value)
        y, h = ssd.ssd_delta_fwd(*a)
        torch.cuda.synchronize()
        yr, hr = oracle.delta_recurrent(*[to_np(v) for v in a])
        assert err(h, hr) <= 2e-5 and err(y, yr) <= tol(y, dtype)
