"""The learned gate as programs use it: in front of the experts, taught by the
mixture, trained; captured in graphs, on other streams, two at a time, in rooms
that others still use.

What is compared with itself has to be equal; sums of whole numbers and powers
of two are exact.  Values are held to the tolerances of test_gate.py.
"""
import numpy as np
import pytest

import soft_clustering_gb300 as G
from test_gate import U, UT, _f64, _logits, _S, _E, gate_grad_ref, gate_ref, softmax_ref


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def _step(layer, gate, teach, norm, rows, w):
    """One pass of all of it: normalised rows, logits of a matrix, the gate, the
    experts, the teacher, and every gradient."""
    X, dout = rows
    Y = norm.forward(X, w["nw"], w["nb"])
    offsets = w["offsets"]
    logits = w["logit"].forward(Y, offsets, w["Wg"])
    ids, gamma = gate.forward(logits, balance=True)
    out = layer.forward(Y, ids, gamma, w["We"])
    dY, dgamma, dWe = layer.backward(dout, w["We"], weight_dtype=w["We"].dtype)
    dlogits = gate.backward(logits, dgamma, balance=0.01)
    total, _ = teach.step(logits, w["tids"], w["tgamma"], out=dlogits, add=True)
    dWg = w["logit"].backward_weights(dlogits, Y, offsets)
    dY2 = w["logit"].backward_rows(dlogits, offsets, w["Wg"])
    dX, dnw, dnb = norm.backward(dY + dY2, X, w["nw"])
    return dict(out=out, loss=gate.loss, total=total, dlogits=dlogits, dWg=dWg, dWe=dWe, dX=dX, dnw=dnw, dnb=dnb,
                ids=ids, gamma=gamma, logits=logits, dgamma=dgamma)


def _parts(seed=0, N=500, D=64, K=16, d_out=32, m=2):
    import torch
    from soft_clustering_gb300.experts import ExpertProduct, LocalExperts
    from soft_clustering_gb300.gate import Distiller, Gate
    from soft_clustering_gb300.norm import LayerNorm
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    t = torch.bfloat16
    w = dict(nw=1 + 0.1 * rand(D), nb=0.1 * rand(D), Wg=rand(1, K, D) * D ** -0.5, We=rand(K, d_out, D) * D ** -0.5,
             offsets=torch.tensor([0, N], device="cuda"), logit=ExpertProduct(1, D, K, t, N))
    w["tids"] = torch.stack([torch.randperm(K, device="cuda", generator=g)[:3] for _ in range(N)]).to(torch.int32)
    w["tgamma"] = torch.softmax(torch.randn(N, 3, device="cuda", generator=g), 1) * 0.9
    parts = (LocalExperts(N, m, K, D, d_out, t), Gate(N, K, m, t, normalised=True), Distiller(N, K, 3, t),
             LayerNorm(D, t), (rand(N, D), 0.01 * rand(N, d_out)), w)
    return parts


@pytest.mark.gpu
def test_the_layer_together(cuda):
    """Every operator on the outputs of the others, against the restatements on the
    same intermediate values."""
    import torch
    parts = _parts()
    r = _step(*parts)
    gate, w = parts[1], parts[5]
    x = _f64(r["logits"])
    N, K = x.shape
    ids, gamma, lse, p, a = gate_ref(x, 2, None, True)
    assert np.array_equal(r["ids"].cpu().numpy(), ids)
    assert np.abs(_f64(r["gamma"]) - gamma).max() < 1e-5
    share = _f64(gate.share)
    assert np.allclose(share, K * np.bincount(ids.reshape(-1), minlength=K) / (2 * N * N), rtol=1e-6)
    d = gate_grad_ref(p, ids, _f64(r["gamma"]), _f64(r["dgamma"]), share, 0.01, True)
    q = _f64(w["tgamma"]) / _f64(w["tgamma"]).sum(1, keepdims=True)
    t = p.copy()
    tids = w["tids"].cpu().numpy()
    for j in range(3):
        t[np.arange(N), tids[:, j]] -= q[:, j]
    first = d + 0.0
    want = first + t / N
    # rounded to bf16 twice: the gate's gradient, then the sum
    bound = UT["bf16"] * (np.abs(first) + np.abs(want)) * 1.01 + 1e-6 * (p + q.max()) / N + 1e-5 * np.abs(first)
    assert (np.abs(_f64(r["dlogits"]) - want) <= bound).all()
    kl = (q * (np.log(q) - np.log(np.take_along_axis(p, tids, 1)))).sum(1).mean()
    assert abs(float(r["total"]) - kl) < 1e-5
    for k in ("out", "dWg", "dWe", "dX", "dnw", "dnb"):
        assert torch.isfinite(r[k].float()).all(), k


@pytest.mark.gpu
def test_captured_in_a_graph(cuda):
    """The whole step captured once and replayed on new rows, equal to the bit to
    the step run as it is."""
    import torch
    parts = _parts(1)
    rows, w = parts[4], parts[5]
    _step(*parts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = _step(*parts)
    other = _parts(2)
    for replay in range(2):
        rows[0].copy_(other[4][0] * (replay + 1))
        w["tids"].copy_(other[5]["tids"])
        w["tgamma"].copy_(other[5]["tgamma"])
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in kept.items()}
        fresh = _parts(1)
        fresh[4][0].copy_(rows[0])
        fresh[5]["tids"].copy_(w["tids"])
        fresh[5]["tgamma"].copy_(w["tgamma"])
        want = _step(*fresh)
        for k in want:
            assert torch.equal(got[k], want[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("K", [64, 300, 5000, 40000])
def test_two_at_once_on_two_streams(cuda, K):
    """Objects of their own on streams of their own, made and used while the
    others run, and kept until that work is done."""
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    from soft_clustering_gb300.norm import LayerNorm
    N = 200
    rng = np.random.default_rng(K)
    L = [_logits(rng, N, K, "bf16", plain=True) for _ in range(2)]
    X = [torch.randn(N, 512, device="cuda") for _ in range(2)]

    kept = []

    def run(i, stream):
        g, d, n = Gate(N, K, 2, L[i].dtype), Distiller(N, K, 2, L[i].dtype), LayerNorm(512, torch.float32)
        kept.extend((g, d, n))
        ids, gamma = g.forward(L[i], balance=True, stream=stream)
        grad = g.backward(L[i], gamma, balance=0.5, stream=stream)
        total, grad = d.step(L[i], ids, gamma, out=grad, add=True, stream=stream)
        Y = n.forward(X[i], stream=stream)
        return [ids, gamma, g.lse, g.counts, g.mass, g.loss, total, grad, Y, *n.backward(Y, X[i], stream=stream)]

    want = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
    got = [run(i, s) for i, s in enumerate(streams)] + [run(0, streams[1].cuda_stream)]
    torch.cuda.synchronize()
    for a, b in zip(want + [want[0]], got):
        for p, q in zip(a, b):
            assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [3, 8, 24, 100, 256, 777, 1024, 3000, 9000, 20000])
def test_neighbours_are_left_as_they_were(cuda, K, dtype):
    """Outputs between words that belong to others, of every form: nothing before
    the first and behind the last row is written."""
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    from soft_clustering_gb300.norm import LayerNorm
    rng = np.random.default_rng(K)
    N, m = 37, 2
    L = _logits(rng, N, K, dtype)
    g, d, n = Gate(N, K, m, L.dtype), Distiller(N, K, m, L.dtype), LayerNorm(K, L.dtype)

    def room(shape, t, pad):
        """A view of this shape with `pad` others' elements on either side."""
        count = int(np.prod(shape))
        whole = torch.full((count + 2 * pad,), 7, dtype=t, device="cuda")
        return whole, whole[pad:pad + count].view(shape)

    for pad in (16, 1):
        ids, gamma = g.forward(L)
        wide = [room((N, m), torch.int32, pad), room((N, m), torch.float32, pad), room((N,), torch.float32, pad)]
        G.gmm_gate(L, g.xdtype, N, K, m, 0, None, wide[0][1], wide[1][1], wide[2][1], None, None, None, None, None, 0)
        assert torch.equal(wide[0][1], ids) and torch.equal(wide[1][1], gamma) and torch.equal(wide[2][1], g.lse)
        out = [room((N, K), L.dtype, pad) for _ in range(4)]
        g.backward(L, gamma, out=out[0][1])
        d.step(L, ids, gamma, out=out[1][1])
        n.forward(L, out=out[2][1])
        n.backward(L, L, out=out[3][1])
        for whole, view in wide + out:
            assert (whole[:pad] == 7).all() and (whole[-pad:] == 7).all()


@pytest.mark.gpu
def test_inputs_written_again_and_outputs_kept(cuda):
    """What a call returned stays until the object's next call, whatever becomes of
    its inputs."""
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    rng = np.random.default_rng(0)
    L = _logits(rng, 300, 200, "bf16", plain=True)
    keep = L.clone()
    g, d = Gate(300, 200, 2, L.dtype), Distiller(300, 200, 2, L.dtype)
    ids, gamma = g.forward(L, balance=True)
    total, grad = d.step(L, ids, gamma)
    torch.cuda.synchronize()
    was = [t.clone() for t in (ids, gamma, g.lse, g.mass, total, grad)]
    L.fill_(float("nan"))
    torch.cuda.synchronize()
    for a, b in zip(was, (ids, gamma, g.lse, g.mass, total, grad)):
        assert torch.equal(a, b)
    # a forward that is refused leaves no backward pass
    with pytest.raises(ValueError):
        g.forward(keep.float())
    g.backward(keep, gamma)  # refused before anything changed
    g.forward(keep)
    with pytest.raises(RuntimeError, match="balance"):
        g.backward(keep, gamma, balance=0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_offsets_past_32_bits(cuda, dtype):
    """Rows behind the first 2^32 bytes and elements: the last ones equal those of a
    call of their own, of enough rows that each is worked on in the same form (few
    long ones are shared by blocks, whose sums are added up in another order)."""
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    from soft_clustering_gb300.norm import LayerNorm
    R = 320
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    for N, K in ((4_200_000, 1024), (131_100, 32768)):
        if torch.cuda.mem_get_info()[0] < 6 * N * K * 2 / 2:
            pytest.skip("needs memory")
        L = torch.zeros(N, K, dtype=t, device="cuda")
        last = torch.randn(R, K, device="cuda").to(t)
        L[-R:] = last
        gate, small = Gate(N, K, 2, t), Gate(R, K, 2, t)
        ids, gamma = gate.forward(L)
        want = small.forward(last)
        assert torch.equal(ids[-R:], want[0]) and torch.equal(gamma[-R:], want[1])
        dg = torch.randn(N, 2, device="cuda")
        out = gate.backward(L, dg)
        assert torch.equal(out[-R:], small.backward(last, dg[-R:].contiguous()))
        a, b = Distiller(N, K, 2, t, scale=1.0), Distiller(R, K, 2, t, scale=1.0)
        a.step(L, ids, gamma, out=out)
        assert torch.equal(out[-R:], b.step(last, *want)[1]) and torch.equal(a.rows[-R:], b.rows)
        norm = LayerNorm(K, t)
        norm.forward(L, out=out)
        assert torch.equal(out[-R:], norm.forward(last))
        del L, out, gate, a, ids, gamma, dg
        torch.cuda.empty_cache()


@pytest.mark.gpu
def test_gradient_against_differences_of_the_kernels(cuda):
    """The kernels' own losses, in fp32, against their gradients along a direction.

    A central difference with step h of a loss near L in fp32 is off by 2^-22 L / h
    from rounding and by h^2 times a third derivative of the order of the loss:
    with h = 2^-6 and L of 1 to 10 below 2^-9 relative to the loss."""
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    N, K = 50, 40
    L = torch.randn(N, K, device="cuda", generator=g)
    v = torch.randn(N, K, device="cuda", generator=g)
    v /= v.norm()
    ids = torch.stack([torch.randperm(K, device="cuda", generator=g)[:4] for _ in range(N)]).to(torch.int32)
    vals = torch.randn(N, 4, device="cuda", generator=g)
    h = 2.0 ** -6
    d = Distiller(N, K, 4, torch.float32, teacher="logits", temperature=2.0, scale=1.0 / 16)
    loss = lambda x: float(d.loss(x, ids, vals))  # noqa: E731
    grad = d.step(L, ids, vals)[1]
    assert abs((loss(L + h * v) - loss(L - h * v)) / (2 * h) - float((grad * v).sum())) < 2 ** -9 * (1 + loss(L))
    # the balance loss with the entries held: their share from the gate, the mass from the moved logits
    gate, moved = Gate(N, K, 2, torch.float32), Gate(N, K, 2, torch.float32)
    gate.forward(L, balance=True)
    share = gate.share.double()

    def balance(x):
        moved.forward(x, balance=True)
        return float((share * moved.mass.double()).sum())

    grad = gate.backward(L, balance=1.0)
    assert abs((balance(L + h * v) - balance(L - h * v)) / (2 * h) - float((grad * v).sum())) < 2 ** -9


@pytest.mark.gpu
def test_example_runs(cuda):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "learned_gate.py")
    spec = importlib.util.spec_from_file_location("learned_gate", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, used = mod.train(N=2000, D=32, K=8, d_out=16, steps=6, teach=3, log=None)
    assert len(losses) == 6 and np.isfinite(losses).all()
    assert used.sum() == 2 * 2000
