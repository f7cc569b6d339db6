"""Rows that are streamed by a block, many of them and with padding anywhere.

A share 1 / K of equal logits is within two units of 2^-24 (exp2(0) = 1 and whole
sums below 2^24 are exact, the reciprocal is within one unit in the last place),
its N-fold sum within one more for each rounding to 32 bits that is left: that of
a stretch of rows, and the result's.
"""
import numpy as np
import pytest

from test_gate import U, _f64, _logits


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,K", [("f16", 8201), ("bf16", 16392), ("f32", 8196), ("f32", 8201)])
def test_mass_of_many_rows(cuda, dtype, K):
    import torch
    from soft_clustering_gb300.gate import Gate
    N = 40000
    t = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    L = torch.zeros(N, K, dtype=t, device="cuda")
    live = torch.arange(N, device="cuda") % 5 != 4
    g = Gate(N, K, 2, t)
    g.forward(L, live=live, balance=True)
    rows = int(live.sum())
    assert (np.abs(_f64(g.mass) / (rows / K) - 1) <= 6 * U).all()
    assert abs(float(g.loss) - 1) <= 8 * U  # even mass, and the entries' shares sum to K / rows
    assert g.counts.tolist()[:3] == [rows, rows, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 20000), (2, 40001), (70, 20001), (400, 17000), (1000, 32768), (5, 65536)])
def test_rows_left_out_of_a_stream(cuda, N, K, dtype):
    """Padding first, last, in runs, everywhere: the rows that count are as they are
    by themselves, bit for bit, the others zeros, or untouched where a gradient is
    added."""
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    rng = np.random.default_rng(N + K)
    m = 3
    L = _logits(rng, N, K, dtype, plain=True)
    ids = torch.from_numpy(rng.integers(0, K, (N, m)).astype(np.int32)).cuda()
    vals = torch.from_numpy(rng.random((N, m)).astype(np.float32)).cuda()
    dg = torch.from_numpy(rng.standard_normal((N, m)).astype(np.float32)).cuda()
    base = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).to(L.dtype).cuda()
    make = lambda: (Gate(N, K, m, L.dtype), Distiller(N, K, m, L.dtype, scale=0.5))  # noqa: E731
    g, d = make()
    want_ids, want_gamma = g.forward(L, balance=True)
    share = g.share.clone()
    want_grad = g.backward(L, dg, balance=0.5)
    _, want_step = d.step(L, ids, vals)
    want_rows = d.rows.clone()
    _, want_add = d.step(L, ids, vals, out=base.clone(), add=True)
    n = np.arange(N)
    for on in (n % 10 != 3, n >= N // 2, n < N // 2, n % 300 < 7, rng.random(N) < 0.1, n < 0, n == N - 1, n >= 0):
        live = torch.from_numpy(on).cuda()
        off = ~live
        poisoned = L.clone()
        poisoned[off] = float("nan")
        g2, d2 = make()
        i2, gam2 = g2.forward(poisoned, live=live, balance=True)
        assert torch.equal(i2[live], want_ids[live]) and torch.equal(gam2[live], want_gamma[live])
        assert (i2[off] == -1).all() and not gam2[off].any()
        g2.share.copy_(share)  # of all rows: the gradient's rows are then the same
        grad = g2.backward(poisoned, dg, live=live, balance=0.5)
        assert torch.equal(grad[live], want_grad[live]) and not grad[off].any()
        w = live.float()
        total, step = d2.step(poisoned, ids, vals, weights=w)
        assert torch.equal(step[live], want_step[live]) and not step[off].any()
        assert torch.equal(d2.rows[live], want_rows[live]) and not d2.rows[off].any()
        assert abs(float(total) - 0.5 * float(d2.rows.double().sum())) <= 4 * U * abs(float(total))
        d2.loss(poisoned, ids, vals, weights=w)
        assert torch.equal(d2.rows[live], want_rows[live]) and not d2.rows[off].any()
        out = base.clone()
        d2.step(poisoned, ids, vals, weights=w, out=out, add=True)
        assert torch.equal(out[live], want_add[live]) and torch.equal(out[off], base[off])
