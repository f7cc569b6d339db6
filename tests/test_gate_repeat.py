"""The gate, distillation and layer norm give the same bits for the same inputs,
call after call, whatever else the device does."""
import numpy as np
import pytest

from test_gate import _logits


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def bits(t):
    """A tensor's bytes, so that NaN and the sign of zero count."""
    import torch
    return t.contiguous().reshape(-1).view(torch.uint8)


def test_bits_tell_values_apart():
    import torch
    a = torch.tensor([1.0, float("nan"), 0.0])
    b = torch.tensor([1.0, float("nan"), -0.0])
    assert torch.equal(bits(a), bits(a.clone())) and not torch.equal(bits(a), bits(b))
    assert not torch.equal(bits(a), bits(torch.tensor([1.0 + 2.0 ** -23, float("nan"), 0.0])))


# every form of row; more rows than the blocks of one wave take at a time
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(30001, 8), (20001, 64), (20000, 61), (9001, 256), (9000, 1000), (5000, 1024),
                                 (3000, 1001), (2000, 4096), (700, 9001), (400, 20000), (400, 40001), (9, 50257)])
def test_bits_repeat(cuda, N, K, dtype):
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    from soft_clustering_gb300.norm import LayerNorm
    L = _logits(np.random.default_rng(N), N, K, dtype)
    live = torch.arange(N, device="cuda") % 7 != 3
    w = live.float() * 1.5
    busy, junk = torch.cuda.Stream(), torch.ones(1 << 24, device="cuda")
    first = None
    for turn in range(4):
        if turn % 2:  # beside others' work, which moves blocks about
            with torch.cuda.stream(busy):
                for _ in range(20):
                    junk.mul_(1.0)
        g, d = Gate(N, K, 2, L.dtype), Distiller(N, K, 2, L.dtype, temperature=2.0)
        out = {}
        out["ids"], out["gamma"] = g.forward(L, live=live, balance=True)
        for k in ("lse", "counts", "mass", "share", "loss"):
            out[k] = getattr(g, k)
        out["dL"] = g.backward(L, out["gamma"], live=live, balance=0.1)
        out["total"], out["dL2"] = d.step(L, out["ids"], out["gamma"], weights=w, out=out["dL"].clone(), add=True)
        out["rows"] = d.rows
        if K <= 32768:
            n = LayerNorm(K, L.dtype)
            X = torch.where(torch.isfinite(L), L, 0.0).clamp_(-100, 100)
            out["Y"] = n.forward(X)
            out["dX"], out["dw"], out["db"] = n.backward(out["Y"], X)
        out = {k: bits(t) for k, t in out.items()}
        torch.cuda.synchronize()
        first = first or out
        for k in first:
            assert torch.equal(first[k], out[k]), (turn, k)
