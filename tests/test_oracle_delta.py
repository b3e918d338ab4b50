"""The fp64 oracle of the gated delta rule and of the norms around its block, tied to something other
than itself: central differences of the forward for every gradient, closed forms, and the chunked
form (the triangular inverse and the carried state) that the tensor-core path evaluates."""
import numpy as np
import pytest

import oracle


def draw(seed, B=2, L=9, H=4, P=3, G=2, N=5):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, L, G, N))
    return dict(x=r.standard_normal((B, L, H, P)), g=-r.uniform(0.01, 1.0, (B, L, H)), beta=r.uniform(0.05, 0.95, (B, L, H)),
                Bm=k / np.linalg.norm(k, axis=-1, keepdims=True), Cm=r.standard_normal((B, L, G, N)) / np.sqrt(N),
                h0=r.standard_normal((B, H, P, N)))


def differences(f, a, i, h):
    up, down = a.copy(), a.copy()
    up.flat[i] += h
    down.flat[i] -= h
    return (f(up) - f(down)) / (2 * h)


@pytest.mark.parametrize("seed", [0, 1])
def test_delta_gradients_by_differences(seed):
    d = draw(seed)
    r = np.random.default_rng(100 + seed)
    dy, dh = r.standard_normal(d["x"].shape), r.standard_normal(d["h0"].shape)
    grads = oracle.delta_backward(*d.values(), dy, dh)
    # rounding of the loss over the step against the step's own error: 1e-16 / 1e-5 and 1e-10
    for name, key in (("x", "dx"), ("g", "dg"), ("beta", "dbeta"), ("Bm", "dB"), ("Cm", "dC"), ("h0", "dh0")):
        def loss(v):
            y, h = oracle.delta_recurrent(**{**d, name: v})
            return float(np.sum(dy * y) + np.sum(dh * h))
        got = np.array([differences(loss, d[name], i, 1e-5) for i in range(d[name].size)])
        assert np.max(np.abs(got - grads[key].ravel())) <= 1e-7 * max(1.0, np.max(np.abs(got))), key


def test_delta_is_a_plain_memory_with_orthonormal_keys():
    """Orthonormal keys, beta = 1, no decay: the state holds x_t under key t, and a query of key s
    returns x_s exactly once it was written; a second write of the same key replaces the first."""
    r = np.random.default_rng(3)
    N = 6
    K = np.linalg.qr(r.standard_normal((N, N)))[0]
    order = [0, 1, 2, 3, 1, 4, 5]
    x = r.standard_normal((1, len(order), 1, 2))
    k = K[order].reshape(1, len(order), 1, N)
    one = np.ones((1, len(order), 1))
    _, S = oracle.delta_recurrent(x, 0 * one, one, k, k)
    last = {s: i for i, s in enumerate(order)}
    for s in range(N):
        np.testing.assert_allclose(S[0, 0] @ K[s], x[0, last[s], 0], atol=1e-12)


def test_delta_without_write_only_decays_and_infinite_decay_clears():
    d = draw(5)
    _, h = oracle.delta_recurrent(d["x"], d["g"], 0 * d["beta"], d["Bm"], d["Cm"], d["h0"])
    np.testing.assert_allclose(h, np.exp(d["g"].sum(1))[..., None, None] * d["h0"], rtol=1e-12)
    g = d["g"].copy()
    g[:, 4] = -np.inf
    y, h = oracle.delta_recurrent(d["x"], g, d["beta"], d["Bm"], d["Cm"], d["h0"])
    tail = {k: v[:, 4:] for k, v in d.items() if k != "h0"}
    y2, h2 = oracle.delta_recurrent(**tail)
    np.testing.assert_allclose(h, h2, rtol=1e-12)
    np.testing.assert_allclose(y[:, 4:], y2, rtol=1e-12)


@pytest.mark.parametrize("chunk", [1, 4, 9, 16])
def test_delta_chunked_form(chunk):
    """With cum the cumulated log decay in a chunk, E_ij = exp(cum_i - cum_j), M = tril(K K^T o E, -1) and
    W the strictly lower solution of W = -M (I + diag(beta) W):
      err = R + W (beta R),  R = X - exp(cum) K S^T,  u = beta err,
      y = exp(cum) Q S^T + tril(Q K^T o E) u,  S <- exp(cum_end) S + u^T (exp(cum_end - cum) K),
    and in reverse, for the leaving cotangent D, with F = tril(Q K^T o E)^T dy + (exp(cum_end - cum) K) D^T:
      z = F + W^T (beta F),  dx = beta z,  dbeta_i = z_i.err_i,
      D <- exp(cum_end) D + dy^T (exp(cum) Q) - dx^T (exp(cum) K)."""
    d = draw(7, L=21)
    r = np.random.default_rng(8)
    dy, dh = r.standard_normal(d["x"].shape), r.standard_normal(d["h0"].shape)
    y_ref, h_ref = oracle.delta_recurrent(**d)
    ref = oracle.delta_backward(*d.values(), dy, dh)
    Bsz, L, H, P = d["x"].shape
    for b in range(Bsz):
        for h in range(H):
            x, g, beta = d["x"][b, :, h], d["g"][b, :, h], d["beta"][b, :, h]
            k, q = d["Bm"][b, :, h // 2], d["Cm"][b, :, h // 2]
            S, parts = d["h0"][b, h], []
            for t0 in range(0, L, chunk):
                t = slice(t0, min(L, t0 + chunk))
                cum = np.cumsum(g[t])
                n = len(cum)
                E = np.exp(np.tril(cum[:, None] - cum[None, :]))
                M = np.tril(k[t] @ k[t].T * E, -1)
                W = np.zeros((n, n))
                for i in range(n):
                    W[i] = -M[i] @ (np.eye(n) + beta[t, None] * W)
                R = x[t] - np.exp(cum)[:, None] * (k[t] @ S.T)
                err = R + W @ (beta[t, None] * R)
                u = beta[t, None] * err
                PQ = np.tril(q[t] @ k[t].T * E)
                parts.append((t, cum, W, PQ, err))
                np.testing.assert_allclose(np.exp(cum)[:, None] * (q[t] @ S.T) + PQ @ u, y_ref[b, t, h], atol=1e-11)
                S = np.exp(cum[-1]) * S + u.T @ (np.exp(cum[-1] - cum)[:, None] * k[t])
            np.testing.assert_allclose(S, h_ref[b, h], atol=1e-11)
            D = dh[b, h]
            for t, cum, W, PQ, err in reversed(parts):
                F = PQ.T @ dy[b, t, h] + (np.exp(cum[-1] - cum)[:, None] * k[t]) @ D.T
                z = F + W.T @ (beta[t, None] * F)
                np.testing.assert_allclose(beta[t, None] * z, ref["dx"][b, t, h], atol=1e-10)
                np.testing.assert_allclose((z * err).sum(1), ref["dbeta"][b, t, h], atol=1e-10)
                D = (np.exp(cum[-1]) * D + dy[b, t, h].T @ (np.exp(cum)[:, None] * q[t])
                     - (beta[t, None] * z).T @ (np.exp(cum)[:, None] * k[t]))
            np.testing.assert_allclose(D, ref["dh0"][b, h], atol=1e-10)


@pytest.mark.parametrize("scale,residual", [(True, True), (False, True), (True, False), (False, False)])
def test_add_rmsnorm_gradients_by_differences(scale, residual):
    r = np.random.default_rng(11)
    rows, dim, eps = 3, 7, 1e-5
    v = {"x": r.standard_normal((rows, dim)), "w": r.standard_normal(dim)}
    if residual:
        v["res"] = r.standard_normal((rows, dim))
    if scale:
        v["scale"] = r.standard_normal(dim)
    do, dr = r.standard_normal((rows, dim)), r.standard_normal((rows, dim))

    def forward(v):
        return oracle.add_rmsnorm(v["x"], v.get("res"), v["w"], scale=v.get("scale"), eps=eps)

    got = oracle.add_rmsnorm_backward(forward(v)[0], v["w"], do, dr, x=v["x"], scale=v.get("scale"), eps=eps)
    for name, key in (("x", "dx"), ("w", "dw"), ("res", "dres"), ("scale", "dscale")):
        if name not in v:
            continue
        def loss(a):
            res, out = forward({**v, name: a})
            return float(np.sum(do * out) + np.sum(dr * res))
        want = np.array([differences(loss, v[name], i, 1e-5) for i in range(v[name].size)])
        assert np.max(np.abs(want - got[key].ravel())) <= 1e-7 * max(1.0, np.max(np.abs(want))), key


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("ngroups", [1, 3])
def test_gate_norm_gradients_by_differences(gate_first, ngroups):
    r = np.random.default_rng(13)
    v = {k: r.standard_normal((4, 12)) for k in ("y", "z")} | {"w": r.standard_normal(12)}
    do = r.standard_normal((4, 12))
    fwd = oracle.gated_rmsnorm if gate_first else oracle.norm_gate
    got = oracle.gate_norm_backward(v["y"], v["z"], v["w"], do, ngroups=ngroups, eps=1e-5, gate_first=gate_first)
    for name, key in (("y", "dy"), ("z", "dz"), ("w", "dw")):
        def loss(a):
            u = {**v, name: a}
            return float(np.sum(do * fwd(u["y"], u["z"], u["w"], ngroups=ngroups, eps=1e-5)))
        want = np.array([differences(loss, v[name], i, 1e-5) for i in range(v[name].size)])
        assert np.max(np.abs(want - got[key].ravel())) <= 1e-7 * max(1.0, np.max(np.abs(want))), key


def test_norm_gate_by_hand():
    """One row, two groups, eps = 0: each group has unit mean square before the weight and the gate."""
    y = np.array([[3.0, 4.0, 0.5, -0.5]])
    z = np.array([[0.0, 30.0, 30.0, 30.0]])  # silu: 0 and 30
    out = oracle.norm_gate(y, z, np.ones(4), ngroups=2, eps=0.0)
    np.testing.assert_allclose(out, [[0.0, 30 * 4 / np.sqrt(12.5), 30.0, -30.0]], rtol=1e-12)
