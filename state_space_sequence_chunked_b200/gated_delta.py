"""The gated-delta mixer and block forward: the Mamba-2 mixer's order of operations (mamba2.py) with
the gated delta rule in the place of the SSD layer, keys and queries of unit length, and the norm
before the gate, one group per head.

    block:  residual, n = ssd_add_rmsnorm(x, residual)      libssd kernel
    mixer:  row = n in_proj^T                               plain GEMM (cuBLAS)  [B, L, 2HP + 2GN + 2H]
            x, B, C, dt = ssd_conv_split(...)               libssd kernel
            B, C = ssd_add_rmsnorm(B), ssd_add_rmsnorm(C)   libssd kernel, rows of N scaled to length 1
                                                            and N^-1/2
            y, h_final = ssd_delta_fwd(x, A dt, sigmoid(beta), B, C)   libssd kernels
            o = ssd_norm_gate(y, z)                         libssd kernel
            out = o out_proj^T                              plain GEMM (cuBLAS)  [B, L, d_model]
"""
from __future__ import annotations

import dataclasses

import torch

from . import _binding as ssd


@dataclasses.dataclass
class DeltaConfig:
    d_model: int
    nheads: int
    headdim: int
    ngroups: int
    dstate: int
    conv_width: int = 4
    eps: float = 1e-5
    key_eps: float = 1e-6  # added to the squared length of keys and queries

    @property
    def d_inner(self) -> int:
        return self.nheads * self.headdim

    @property
    def d_in_proj(self) -> int:
        return 2 * self.d_inner + 2 * self.ngroups * self.dstate + 2 * self.nheads


@dataclasses.dataclass
class DeltaWeights:
    in_proj: torch.Tensor    # [d_in_proj, d_model], input dtype: rows z | x B C | dt_raw | beta_raw
    conv_w: torch.Tensor     # [H*P + 2*G*N, W] fp32
    conv_b: torch.Tensor     # [H*P + 2*G*N] fp32
    dt_bias: torch.Tensor    # [H] fp32
    A: torch.Tensor          # [H] fp32, negative
    norm_w: torch.Tensor     # [H*P] fp32
    out_proj: torch.Tensor   # [d_model, H*P], input dtype


def mixer_fwd(u: torch.Tensor, w: DeltaWeights, cfg: DeltaConfig, h0=None):
    """u [B, L, d_model] -> (out [B, L, d_model], h_final [B, H, P, N])."""
    H, HP, GN, N = cfg.nheads, cfg.d_inner, cfg.ngroups * cfg.dstate, cfg.dstate
    row = torch.matmul(u, w.in_proj.t())
    z, xbc = row[..., :HP], row[..., HP:2 * HP + 2 * GN]
    dt_raw, beta = row[..., 2 * HP + 2 * GN:2 * HP + 2 * GN + H], torch.sigmoid(row[..., 2 * HP + 2 * GN + H:])
    s = ssd.ssd_conv_split(xbc, dt_raw, w.conv_w, w.conv_b, w.dt_bias, nheads=H, headdim=cfg.headdim,
                           ngroups=cfg.ngroups, dstate=N)
    unit = torch.full((N,), N ** -0.5, dtype=torch.float32, device=u.device)  # rms 1 -> length 1
    _, keys = ssd.ssd_add_rmsnorm(s["B"], None, unit, eps=cfg.key_eps / N, want_res=False)
    _, queries = ssd.ssd_add_rmsnorm(s["C"], None, unit * N ** -0.5, eps=cfg.key_eps / N, want_res=False)
    y, hf = ssd.ssd_delta_fwd(s["x"], (s["dt"] * w.A).to(u.dtype), beta, keys, queries, h0)
    o = ssd.ssd_norm_gate(y.view(*u.shape[:2], HP), z, w.norm_w, ngroups=H, eps=cfg.eps)
    return torch.matmul(o, w.out_proj.t()), hf


def block_fwd(x: torch.Tensor, residual, w: DeltaWeights, cfg: DeltaConfig, pre_norm_w, *, scale=None, h0=None):
    """x, the last block's output, joins the residual stream (None: it starts it) with its per-channel
    scale, and the mixer runs on the stream's norm. Returns (out, residual, h_final); the stream is
    fp32."""
    if residual is None:
        residual = torch.zeros(x.shape, dtype=torch.float32, device=x.device)
    residual, n = ssd.ssd_add_rmsnorm(x, residual, pre_norm_w, scale=scale, eps=cfg.eps)
    out, hf = mixer_fwd(n, w, cfg, h0)
    return out, residual, hf
