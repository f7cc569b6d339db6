"""Layer norm and its gradients (gmm_layer_norm, gmm_layer_norm_grad).

CPU: refusals, and the 64-bit restatement against differences.  GPU: the kernels
against the restatement.

Tolerances, from the operations alone (u = 2^-24, uT the unit roundoff of the
type; fp16 results below 2^-14 also lose up to 2^-25).  Sums over a row: at most
300 terms one after another or in a tree, 300 u of the sum of their sizes.
  c = x - mean: 2 u |mean| (the mean held in 32 bits) + 2 u |x - mean| + 302 u of
  the row's mean |x - mean|
  1 / sigma: (310 u + 2 c / sigma) of itself, sigma^2 = var + eps; h = c / sigma
  sums over N rows: N / 100 + 64 one after another before 64 bits
"""
import numpy as np
import pytest

import soft_clustering_gb300 as G
from test_gate import CODE, SUB, U, UT, _dt, _f64, _misaligned, _near


def norm_ref(x, eps, w, b):
    mean = x.mean(1, keepdims=True)
    s = np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + eps)
    h = (x - mean) / s
    return h * w + b, h, s, mean


def grad_ref(dy, h, s, w):
    g = dy * w
    dx = (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True)) / s
    return dx, (dy * h).sum(0), dy.sum(0)


def test_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, c, w, b = rng.standard_normal((3, 5)), rng.standard_normal((3, 5)), rng.random(5) + 0.5, rng.random(5)
    y, h, s, _ = norm_ref(x, 1e-2, w, b)
    dx, dw, db = grad_ref(c, h, s, w)
    loss = lambda x, w, b: (c * norm_ref(x, 1e-2, w, b)[0]).sum()  # noqa: E731
    args = [x, w, b]
    for n, d in enumerate((dx, dw, db)):
        for i in np.ndindex(*args[n].shape):
            lo, hi = [v.copy() for v in args], [v.copy() for v in args]
            lo[n][i] -= 1e-5
            hi[n][i] += 1e-5
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - d[i]) < 1e-7


@pytest.fixture(scope="module")
def lib():
    from soft_clustering_gb300 import build
    build.build()
    return G.lib()


def test_refusals_before_anything_is_queued(lib):
    bad, P, big = G.GMM_ERR_INVALID_ARG, 4096, 1 << 40

    def each(f, args, wrong):
        for i, v in wrong:
            a = list(args)
            a[i] = v
            assert f(*a) == bad, (f.__name__, i, v)

    fwd = [P, 1, 10, 64, 1e-5, P, P, 1, P, None]
    each(lib.gmm_layer_norm, fwd, [(0, None), (0, P + 1), (1, 3), (2, -1), (2, 2 ** 31), (3, 0), (4, -1.0),
                                   (4, float("nan")), (4, float("inf")), (5, P + 1), (6, P + 1), (7, 2), (7, -1),
                                   (8, None), (8, P + 1)])
    fwd[3] = 32769
    assert lib.gmm_layer_norm(*fwd) == G.GMM_ERR_UNSUPPORTED
    bwd = [P, P, 1, 10, 64, 1e-5, P, 0, P, P, P, P, big, None]
    each(lib.gmm_layer_norm_grad, bwd, [(0, None), (0, P + 1), (1, None), (1, P + 1), (2, 3), (3, -1), (4, 0),
                                        (5, -1.0), (5, float("nan")), (6, P + 2), (7, 2), (8, P + 1), (9, None),
                                        (9, P + 2), (10, None), (10, P + 2), (11, None), (11, P + 128)])
    bwd[12] = G.gmm_layer_norm_ws_bytes(64) - 1
    assert lib.gmm_layer_norm_grad(*bwd) == G.GMM_ERR_WORKSPACE
    bwd[4] = 32769
    assert lib.gmm_layer_norm_grad(*bwd) == G.GMM_ERR_UNSUPPORTED
    for D in (0, -1, 32769):
        assert G.gmm_layer_norm_ws_bytes(D) == 0
    assert lib.gmm_layer_norm(None, 0, 0, 8, 0.0, None, None, 0, None, None) == G.GMM_OK
    assert lib.gmm_layer_norm_grad(None, None, 0, 0, 8, 0.0, None, 0, None, None, None, None, 0, None) == G.GMM_OK


def test_python_refusals(monkeypatch):
    import torch
    from soft_clustering_gb300 import norm
    for make in (lambda: norm.LayerNorm(8, torch.float16, device="cpu"), lambda: norm.LayerNorm(0, torch.float16),
                 lambda: norm.LayerNorm(40000, torch.float16), lambda: norm.LayerNorm(8, torch.float64),
                 lambda: norm.LayerNorm(8, torch.float16, weight_dtype=torch.bfloat16),
                 lambda: norm.LayerNorm(8, torch.float32, weight_dtype=torch.float16),
                 lambda: norm.LayerNorm(8, torch.float16, eps=-1.0),
                 lambda: norm.LayerNorm(8, torch.float16, eps=float("nan"))):
        with pytest.raises(ValueError):
            make()
    n = object.__new__(norm.LayerNorm)
    n.D, n.dtype, n.weight_dtype, n.device, n._weight = 8, torch.float16, torch.float32, torch.device("cpu"), (8,)
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(8)
    for call in (lambda: n.forward(x.float()), lambda: n.forward(x[0]), lambda: n.forward(x[:, :4]),
                 lambda: n.forward(x, w.half()), lambda: n.forward(x, w, w[:4]), lambda: n.backward(x[:3], x),
                 lambda: n.backward(x, x, w.half()), lambda: n.forward(torch.zeros(8, 4, dtype=torch.float16).T)):
        with pytest.raises(ValueError):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(norm, "_need", lambda t, *a: t)
    n.device = torch.device("cuda", 1)
    for call in (lambda: n.forward(x), lambda: n.backward(x, x)):
        with pytest.raises(ValueError, match="current device"):
            call()


# -------------------------------------------------------------------------- GPU

@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


SIZES = [(1, 1), (5, 2), (700, 3), (9, 7), (1000, 8), (33, 15), (40, 31), (130, 64), (77, 65), (2049, 128),
         (60, 100), (50, 255), (300, 256), (41, 257), (25, 1000), (400, 1024), (1, 1024), (19, 1025), (30, 2048),
         (17, 3001), (200, 4096), (9, 4097), (11, 8192), (7, 10007), (5, 16384), (4, 20000), (3, 32768), (3, 32767)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"),
                                          ("bf16", "f32")])
@pytest.mark.parametrize("N,D", SIZES)
def test_norm(cuda, N, D, dtype, wdtype):
    import torch
    from soft_clustering_gb300.norm import LayerNorm
    rng = np.random.default_rng(N * 13 + D)
    for shifted, affine, eps in ((False, True, 1e-5), (True, True, 1e-3), (False, False, 1e-5)):
        x = rng.standard_normal((N, D)) * rng.random(D) + 0.5 * rng.standard_normal((N, 1))
        if N > 4:
            x[0] = 0.25                       # no spread
            x[1] = 100.0 + 0.5 * x[1]         # far from zero
            x[2] *= 1e-3                      # below eps
            x[3] *= 100.0
        dt, wt = _dt(dtype), _dt(wdtype)
        X = torch.from_numpy(x.astype(np.float32)).to(dt).cuda()
        dY = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32)).to(dt).cuda()
        w = torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).to(wt).cuda()
        b = torch.from_numpy(rng.standard_normal(D).astype(np.float32)).to(wt).cuda()
        if shifted:
            X, dY, w, b = (_misaligned(t) for t in (X, dY, w, b))
        n = LayerNorm(D, dt, eps=eps, weight_dtype=wt)
        x, dy = _f64(X), _f64(dY)
        rw, rb = (_f64(w), _f64(b)) if affine else (np.ones(D), np.zeros(D))
        y, h, s, mean = norm_ref(x, eps, rw, rb)
        uT, sub = UT[dtype], SUB[dtype]
        c = np.abs(x - mean)
        ec = 2 * U * np.abs(mean) + 2 * U * c + 302 * U * c.mean(1, keepdims=True)
        rel = 310 * U + 2 * ec.max(1, keepdims=True) / s
        eh = ec / s + np.abs(h) * (rel + 4 * U)
        args = (w, b) if affine else (None, None)
        out = _misaligned(torch.zeros_like(X)) if shifted else None
        Y = n.forward(X, *args, out=out)
        _near(Y, y, np.abs(rw) * eh + 2 * U * (np.abs(h * rw) + np.abs(y)) + uT * np.abs(y) + sub, "Y")
        dX, dw, db = n.backward(dY, X, args[0], out=_misaligned(torch.zeros_like(X)) if shifted else None)
        rx, rdw, rdb = grad_ref(dy, h, s, rw)
        g, gh = np.abs(dy * rw), np.abs(dy * rw * h)
        mg, mgh = g.mean(1, keepdims=True), gh.mean(1, keepdims=True)
        eb = 304 * U * mgh + (g * eh).mean(1, keepdims=True)
        ex = (4 * U * g + 304 * U * mg + np.abs(h) * eb + (eh + 4 * U * np.abs(h)) * mgh
              + (g + mg + np.abs(h) * mgh) * (rel + 4 * U)) / s
        _near(dX, rx, ex + uT * np.abs(rx) + sub, "dX")
        chain = (N / 100 + 64) * U
        uW, subw = UT[wdtype], SUB[wdtype]
        _near(dw, rdw, (np.abs(dy) * eh).sum(0) + chain * np.abs(dy * h).sum(0) + uW * np.abs(rdw) + subw, "dweight")
        _near(db, rdb, chain * np.abs(dy).sum(0) + uW * np.abs(rdb) + subw, "dbias")
        # the rows' gradient alone, and to the bit again
        alone, none, _ = n.backward(dY, X, args[0], weight_grads=False)
        assert none is None and torch.equal(alone, dX)
        again = n.backward(dY, X, args[0])
        for p, q in zip(again, (dX, dw, db)):
            assert torch.equal(p, q)


@pytest.mark.gpu
@pytest.mark.parametrize("N,D", [(40000, 64), (9000, 1000), (3000, 4096)])
def test_weight_gradient_alone_and_over_many_rows(cuda, N, D):
    """dX left out through the C ABI, and long sums over rows."""
    import torch
    rng = np.random.default_rng(D)
    X = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32)).cuda()
    dY = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32)).cuda()
    dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    ws = torch.empty(G.gmm_layer_norm_ws_bytes(D), dtype=torch.uint8, device="cuda")
    G.gmm_layer_norm_grad(dY, X, G.GMM_F32, N, D, 1e-5, None, G.GMM_F32, None, dw, db, ws, ws.numel())
    x, dy = _f64(X), _f64(dY)
    _, h, s, mean = norm_ref(x, 1e-5, 1.0, 0.0)
    _, rw, rb = grad_ref(dy, h, s, 1.0)
    # the walk of rounding over sums of terms with either sign: 1e-6 of the sum's own size, the square root of N
    assert np.linalg.norm(_f64(dw) - rw) < 1e-6 * np.linalg.norm(rw)
    assert np.linalg.norm(_f64(db) - rb) < 1e-6 * np.linalg.norm(rb)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [5, 128, 1000, 5000])
def test_rows_that_are_not_finite(cuda, D):
    """An infinity or NaN in a row is in no other row."""
    import torch
    from soft_clustering_gb300.norm import LayerNorm
    rng = np.random.default_rng(D)
    X = torch.from_numpy(rng.standard_normal((70, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    n = LayerNorm(D, torch.bfloat16)
    want, grad = n.forward(X), n.backward(X, X, weight_grads=False)[0]
    X2 = X.clone()
    X2[3, 1], X2[60, D - 1] = float("inf"), float("nan")
    got, g2 = n.forward(X2), n.backward(X, X2, weight_grads=False)[0]
    even = [i for i in range(70) if i not in (3, 60)]
    assert torch.equal(got[even], want[even]) and torch.equal(g2[even], grad[even])
    assert torch.isnan(got[[3, 60]]).all() and torch.isnan(g2[[3, 60]]).all()


@pytest.mark.gpu
def test_no_rows(cuda):
    import torch
    from soft_clustering_gb300.norm import LayerNorm
    X = torch.empty(0, 24, dtype=torch.float16, device="cuda")
    n = LayerNorm(24, X.dtype, weight_dtype=torch.float32)
    w = torch.ones(24, device="cuda")
    assert n.forward(X, w, w).shape == (0, 24)
    dX, dw, db = n.backward(X, X, w)
    assert dX.shape == (0, 24) and not dw.any() and not db.any()
