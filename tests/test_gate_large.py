"""The gate and distillation where logits, or logits over a temperature, are large:
rows masked with -1e9 to -1e30 instead of -inf, whole or but for a few components,
values on both sides of where the kernels change how they take an exponent.

Held to test_gate.py's tolerances: those go by an exponent's distance from the
row's largest, whatever the size of both.
"""
import numpy as np
import pytest

from test_gate import (SUB, U, UT, _E, _S, _f64, _misaligned, _near, balance_ref, distill_ref, gate_grad_ref,
                       gate_ref, softmax_ref)

# a lane to a row, lanes of a warp, all of it, a block, streamed; aligned and odd
WIDTHS = [6, 8, 24, 40, 100, 128, 200, 256, 500, 512, 1000, 1024, 1025, 4096, 5000, 8192, 9001, 16384, 20000, 40001]


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def _rows(rng, K, dtype):
    """Rows of such logits, as the type holds them."""
    import torch
    t = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    top = float(torch.finfo(t).max)
    border = 2.0 ** 20 * np.log(2)  # an exponent of base 2 of 2^20
    fills = [f for f in (-1e9, -1e10, -1e30, 1e10, 2e38, -6e4, 6e4) if abs(f) <= top]
    rows = [np.full(K, f) for f in fills]
    for f in fills + [-top]:  # four that are allowed, at either end or anywhere
        for at in (np.arange(4), np.arange(K - 4, K), rng.permutation(K)[:4]):
            r = np.full(K, min(f, -f))
            r[at] = rng.standard_normal(4) * 2
            rows.append(r)
    if top > 1e9:
        rows += [1e6 + rng.standard_normal(K) * 4, rng.standard_normal(K) * 4 - 1e6,
                 border + rng.standard_normal(K) * 3, -border + rng.standard_normal(K) * 3,
                 np.where(np.arange(K) < K // 2, border - 1, border + 1), -1e10 + 4096.0 * rng.integers(0, 3, K)]
    rows += [rng.standard_normal(K) * 2, rng.standard_normal(K) * 50]
    return torch.from_numpy(np.stack(rows).astype(np.float32)).to(t).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", WIDTHS)
def test_gate_of_large_logits(cuda, K, dtype):
    import torch
    from soft_clustering_gb300.gate import Gate
    rng = np.random.default_rng(K)
    m = 4
    for case in range(4):
        normalised, shifted = case & 1, case >= 2
        L = _rows(rng, K, dtype)
        N = L.shape[0]
        if shifted:
            L = _misaligned(L)
        x = _f64(L)
        g = Gate(N, K, m, L.dtype, normalised=bool(normalised))
        ids, gamma = g.forward(L, balance=True)
        rid, rg, rl, p, a = gate_ref(x, m, None, normalised)
        assert np.array_equal(ids.cpu().numpy(), rid), "ids"
        S, E = _S(p, a), _E(a)
        rel = np.take_along_axis(E, rid, 1) + S + 4 * U
        if normalised:
            rel = rel + (rg * rel).sum(1, keepdims=True) + 8 * U
        _near(gamma, rg, rg * rel + 2.0 ** -120, "gamma")
        logs = np.log(np.exp(a).sum(1))
        _near(g.lse, rl, S[:, 0] + 4 * U * (np.abs(rl) + logs) + 4 * U, "lse")
        relp = E + S + 4 * U
        rc, rm, share, loss = balance_ref(rid, p, N)
        assert np.array_equal(g.counts.cpu().numpy(), rc)
        bm = (p * relp).sum(0) + (N / 100 + 64) * U * rm + N * 2.0 ** -120
        _near(g.mass, rm, bm, "mass")
        _near(g.share, share, 2 * U * share, "share")
        _near(_f64(g.loss), np.array([loss]), (share * (bm + 4 * U * rm)).sum() + 2 * U * loss, "loss")
        dg = torch.from_numpy(rng.standard_normal((N, m)).astype(np.float32)).cuda()
        kg, kd, sh = _f64(gamma), _f64(dg), _f64(g.share)
        for coef in (0.3, 0.0):
            got = g.backward(L, dg, balance=coef, out=_misaligned(torch.zeros_like(L)) if shifted else None)
            s = sh if coef else None
            ref = gate_grad_ref(p, rid, kg, kd, s, coef, normalised)
            v = np.abs(kg * kd)
            if normalised:
                v = v + kg * v.sum(1, keepdims=True)
            per = v.sum(1, keepdims=True) + np.zeros((1, K))
            if coef:
                per = per + coef * (sh + (p * sh).sum(1, keepdims=True))
            size = p * per
            for t in range(m):
                size[np.arange(N), rid[:, t]] += v[:, t]
            _near(got, ref, (relp + 2 * S + 340 * U) * size + UT[dtype] * np.abs(ref) + SUB[dtype] + 2.0 ** -126 * per,
                  "dlogits")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", WIDTHS + [50257, 131072])
def test_distill_of_large_logits(cuda, K, dtype):
    """Temperatures that make them larger too.  More rows than few, so that long ones
    belong to blocks, and few."""
    import torch
    from soft_clustering_gb300.gate import Distiller
    rng = np.random.default_rng(K)
    m = 4
    for T, shifted, few in ((1.0, False, False), (0.5, True, False), (2.0 ** -20, False, True), (100.0, False, False)):
        L = _rows(rng, K, dtype)
        if few:
            L = L[torch.from_numpy(rng.permutation(L.shape[0])[:12]).cuda()].contiguous()
        elif K > 8192:  # long rows belong to blocks
            L = L.repeat(3, 1)
        N = L.shape[0]
        if shifted:
            L = _misaligned(L)
        x = _f64(L)
        # the teacher's entries are the row's largest, whose exponents are near
        ids = np.argsort(-x, axis=1, kind="stable")[:, :m].astype(np.int32)
        vals = (0.1 + rng.random((N, m))).astype(np.float32)
        w, scale = np.ones(N), 0.25
        # of logits less their largest, which is the same: 64 bits do not hold 2e38 + log K
        ref, loss, rd, p, q, u, _ = distill_ref(x - x.max(1, keepdims=True), ids, vals.astype(float), "gamma", T, w,
                                                scale)
        _, _, a = softmax_ref(x / T)
        d = Distiller(N, K, m, L.dtype, temperature=T, scale=scale)
        total, got = d.step(L, torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda(),
                            out=_misaligned(torch.zeros_like(L)) if shifted else None)
        S = _S(p, a)
        umax = np.abs(u).max(1, keepdims=True)
        spread = np.abs(u - u.max(1, keepdims=True))
        relq = 16 * U * umax + 4 * U * spread + 2.0 ** -20 + 300 * U
        la = np.where(q > 0, np.abs(np.take_along_axis(a, ids, 1)), 0.0)
        size = 1 + umax[:, 0] + (q * (spread + la)).sum(1) + np.log(np.exp(a).sum(1))
        br = T * T * ((relq * q).sum(1) + S[:, 0] + 64 * U) * size
        _near(d.rows, ref, br, "rows")
        _near(total, np.array([loss]), scale * br.sum() + 2 * U * abs(loss), "loss")
        big = scale * T * p * (_E(a) + S + 4 * U)
        peak = scale * T * q * (relq + 8 * U)
        for t in range(m):
            big[np.arange(N), ids[:, t]] += peak[:, t]
        _near(got, rd, big + 8 * U * scale * T * p + UT[dtype] * np.abs(rd) + SUB[dtype] + 4 * U * np.abs(rd),
              "dlogits")
