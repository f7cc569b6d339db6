"""A mixture of local experts: fit a Gaussian mixture by EM, use its soft
assignment as the gate, and learn one matrix per component by gradient.

The target is piecewise linear: each point's answer comes from the matrix of
the planted component it was drawn from.  One expert per fitted component and
the top-2 responsibilities recover it; one matrix for all points cannot.

    python examples/local_experts.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import soft_clustering_gb300 as G  # noqa: E402
from soft_clustering_gb300.adamw import AdamW  # noqa: E402
from soft_clustering_gb300.experts import LocalExperts  # noqa: E402
from soft_clustering_gb300.torch_api import Assigner, GMMState  # noqa: E402


def planted(N, D, K, d_out, seed, device="cuda"):
    """Points of K well separated clusters, and answers linear within each."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    mu = 4.0 * torch.randn(K, D, device=device, generator=g)
    A = torch.randn(K, d_out, D, device=device, generator=g) * D ** -0.5
    k = torch.randint(0, K, (N,), device=device, generator=g)
    X = (mu[k] + torch.randn(N, D, device=device, generator=g)).to(torch.bfloat16)
    y = torch.bmm(A[k], X.float()[..., None])[..., 0]
    return X, y


def fit_gate(X, K, iters=15):
    """EM from K of the points; top-2 ids and responsibilities of every point."""
    N, D = X.shape
    state = GMMState(N, D, K, G.GMM_COV_DIAG, G.GMM_BF16)
    x = X.float()
    first = [0]  # farthest points first: no two seeds in one cluster
    near = ((x - x[0]) ** 2).sum(1)
    for _ in range(K - 1):
        first.append(int(near.argmax()))
        near = torch.minimum(near, ((x - x[first[-1]]) ** 2).sum(1))
    state.set_params(torch.full((K,), 1.0 / K), x[first], x.var(0).expand(K, D))
    state.opts.var_floor = 1e-4
    state.fit(X, iters, tol=1e-6)
    gate = Assigner(N, D, K, G.GMM_COV_DIAG, G.GMM_BF16, m=2)
    gate.prepare(state.pi.cpu(), state.mu.cpu(), state.cov.cpu())
    gate.assign(X)
    return gate


def train(N=20000, D=64, K=16, d_out=32, steps=150, state_bits=8, seed=0, log=print):
    """Mean squared error before each step."""
    X, y = planted(N, D, K, d_out, seed)
    gate = fit_gate(X, K)
    W = torch.zeros(K, d_out, D, dtype=torch.bfloat16, device=X.device)
    layer = LocalExperts(N, gate.m, K, D, d_out, torch.bfloat16)
    opt = AdamW([W], lr=1e-2, weight_decay=0.0, state_bits=state_bits, master=True,
                rounding="seeded")
    losses = []
    for i in range(steps):
        off = layer.forward(X, gate.ids, gate.gamma, W).float() - y
        losses.append(float(off.square().mean()))
        dout = (off * (2.0 * D / off.numel())).to(torch.bfloat16)
        _, _, dW = layer.backward(dout, W, weight_dtype=torch.float32)
        opt.step([dW])
        if log and i % 25 == 0:
            log("step %4d  mean squared error %.5f" % (i, losses[-1]))
    assert layer.device_status() == G.GMM_OK
    return losses


if __name__ == "__main__":
    out = train()
    print("mean squared error %.5f -> %.5f" % (out[0], out[-1]))
