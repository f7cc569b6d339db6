"""Rows that are streamed: the elements before the first and behind the last
boundary of 16 bytes weigh as much as the others.  Held to test_gate.py's
tolerances, with rows whose logits lie far from zero."""
import numpy as np
import pytest

from test_gate import (SUB, U, UT, _E, _S, _f64, _near, balance_ref, distill_ref, gate_grad_ref, gate_ref,
                       softmax_ref)


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def _rows(rng, K, dtype):
    """Small numbers far from zero, the edges larger than the rest or as large."""
    import torch
    t = {"f32": torch.float32, "f16": torch.float16}[dtype]
    x = np.stack([np.full(K, f) + (n % 2) * rng.standard_normal(K)
                  for n, f in enumerate([-6e4, -6e4, 6e4, 6e4, 40001.0, -50003.0, 777.7, -999.9] * 2)])
    x[8:, :3] += 4
    x[8:, -3:] += 4
    return torch.from_numpy(x.astype(np.float32)).to(t).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("K", [8193, 9001, 16387, 40001])
def test_gate_edges(cuda, K, dtype):
    from soft_clustering_gb300.gate import Gate
    m = 4
    L = _rows(np.random.default_rng(K), K, dtype)
    N = L.shape[0]
    g = Gate(N, K, m, L.dtype)
    ids, gamma = g.forward(L, balance=True)
    rid, rg, rl, p, a = gate_ref(_f64(L), m)
    assert np.array_equal(ids.cpu().numpy(), rid)
    S, E = _S(p, a), _E(a)
    _near(gamma, rg, rg * (np.take_along_axis(E, rid, 1) + S + 4 * U), "gamma")
    _near(g.lse, rl, S[:, 0] + 4 * U * (np.abs(rl) + np.log(np.exp(a).sum(1))) + 4 * U, "lse")
    relp = E + S + 4 * U
    rm = balance_ref(rid, p, N)[1]
    _near(g.mass, rm, (p * relp).sum(0) + (N / 100 + 64) * U * rm, "mass")
    sh = _f64(g.share)
    ref = gate_grad_ref(p, rid, _f64(gamma), np.zeros((N, m)), sh, 0.3, False)
    size = p * 0.3 * (sh + (p * sh).sum(1, keepdims=True))
    _near(g.backward(L, balance=0.3), ref, (relp + 2 * S + 340 * U) * size + UT[dtype] * np.abs(ref) + SUB[dtype], "dL")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("N", [16, 96])
@pytest.mark.parametrize("K", [8193, 16387, 40001, 100001])
def test_distill_edges(cuda, K, N, dtype):
    """Few rows, shared by blocks, and as many as have a block each."""
    import torch
    from soft_clustering_gb300.gate import Distiller
    rng = np.random.default_rng(K)
    L = _rows(rng, K, dtype).repeat(N // 16, 1)
    T = 2.0
    ids = np.tile(np.array([0, 1, K - 1, K // 2], dtype=np.int32), (N, 1))
    vals = np.ones((N, 4), dtype=np.float32)
    d = Distiller(N, K, 4, L.dtype, temperature=T, scale=1.0)
    _, got = d.step(L, torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda())
    x = _f64(L)
    ref, _, rd, p, q, _, _ = distill_ref(x, ids, vals.astype(float), "gamma", T, np.ones(N), 1.0)
    _, _, a = softmax_ref(x / T)
    S = _S(p, a)
    la = np.abs(np.take_along_axis(a, ids, 1))
    relq = 2.0 ** -20 + 300 * U
    _near(d.rows, ref, T * T * (relq + S[:, 0] + 64 * U) * (1 + (q * la).sum(1) + np.log(np.exp(a).sum(1))), "rows")
    big = T * p * (_E(a) + S + 12 * U)
    for t in range(4):
        big[np.arange(N), ids[:, t]] += T * q[:, t] * (relq + 8 * U)
    _near(got, rd, big + (UT[dtype] + 4 * U) * np.abs(rd) + SUB[dtype], "dlogits")
