"""A learned gate for a mixture of local experts: taught by the fitted mixture,
then trained with the experts.

EM fits a Gaussian mixture; its top-2 responsibilities are the teacher of a gate
that answers from a matrix of its own.  For the first steps the gate learns them
(distillation), afterwards it learns from the experts' loss, kept in balance.

    python examples/learned_gate.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import soft_clustering_gb300 as G  # noqa: E402
from soft_clustering_gb300.adamw import AdamW  # noqa: E402
from soft_clustering_gb300.experts import ExpertProduct, LocalExperts  # noqa: E402
from soft_clustering_gb300.gate import Distiller, Gate  # noqa: E402
from soft_clustering_gb300.norm import LayerNorm  # noqa: E402

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from local_experts import fit_gate, planted  # noqa: E402


def train(N=20000, D=64, K=16, d_out=32, steps=200, teach=50, seed=0, log=print):
    """(mean squared error before each step, entries of each component at the end)."""
    X, y = planted(N, D, K, d_out, seed)
    teacher = fit_gate(X, K)
    bf16, dev = torch.bfloat16, X.device
    norm, w, b = LayerNorm(D, bf16), torch.ones(D, dtype=bf16, device=dev), torch.zeros(D, dtype=bf16, device=dev)
    # one component's product is a matrix for all rows: the gate's logits
    logit, all_rows = ExpertProduct(1, D, K, bf16, N), torch.tensor([0, N], device=dev)
    Wg = torch.zeros(1, K, D, dtype=bf16, device=dev)
    We = torch.zeros(K, d_out, D, dtype=bf16, device=dev)
    gate = Gate(N, K, 2, bf16, normalised=True)
    distil = Distiller(N, K, teacher.m, bf16)
    layer = LocalExperts(N, gate.m, K, D, d_out, bf16)
    opt = AdamW([Wg, We, w, b], lr=1e-2, weight_decay=0.0, state_bits=8, master=True, rounding="seeded")
    losses = []
    for i in range(steps):
        Y = norm.forward(X, w, b)
        logits = logit.forward(Y, all_rows, Wg)
        ids, gamma = gate.forward(logits, balance=True)
        off = layer.forward(X, ids, gamma, We).float() - y
        losses.append(float(off.square().mean()))
        dout = (off * (2.0 * D / off.numel())).to(bf16)
        _, dgamma, dWe = layer.backward(dout, We, weight_dtype=torch.float32)
        dlogits = gate.backward(logits, dgamma if i >= teach else None, balance=0.01)
        if i < teach:
            distil.step(logits, teacher.ids, teacher.gamma, out=dlogits, add=True)
        dWg = logit.backward_weights(dlogits, Y, all_rows, out_dtype=torch.float32)
        dY = logit.backward_rows(dlogits, all_rows, Wg)
        _, dw, db = norm.backward(dY, X, w)
        opt.step([dWg, dWe, dw, db])
        if log and i % 25 == 0:
            log("step %4d  mean squared error %.5f  balance %.3f" % (i, losses[-1], float(gate.loss)))
    assert layer.device_status() == logit.device_status() == G.GMM_OK
    return losses, gate.counts.cpu().numpy()


if __name__ == "__main__":
    out, used = train()
    print("mean squared error %.5f -> %.5f; entries of each component %d to %d"
          % (out[0], out[-1], used.min(), used.max()))
