"""A learned gate (gmm_gate, gmm_gate_grad) and distillation (gmm_distill).

CPU: refusals, sizes, and the 64-bit restatements against worked examples and
differences.  GPU: the kernels against the restatements.

Tolerances, from the operations alone (u = 2^-24, uT the unit roundoff of the
type: 0 for fp32, 2^-11 for fp16, 2^-8 for bf16; fp16 results below 2^-14 also
lose up to 2^-25).  Indices and counts are equal.
  e = exp((x - max) / T): the exponent a takes at most four roundings, exp2
  itself at most 2^-21 of its result (tables of a few ulp):
  E(a) = 4 u |a| + 2^-21; below 2^-126 a result may be 0
  sums over a row: at most 300 terms one after another or in a tree, so with
  S = 300 u + sum_k p_k E(a_k) a share p_k is within E(a_k) + S + 4 u
  sums over N rows: N / 100 + 64 one after another before 64 bits
"""
import numpy as np
import pytest

import soft_clustering_gb300 as G

U = 2.0 ** -24
UT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}
CODE = {"f32": G.GMM_F32, "f16": G.GMM_F16, "bf16": G.GMM_BF16}


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


# ------------------------------------------------------- restatements, 64 bits

def softmax_ref(x):
    """p, lse, and x - max (a row of -inf: zeros, -inf, 0)."""
    with np.errstate(all="ignore"):
        top = x.max(1, keepdims=True)
        low = np.where(np.isneginf(top), 0.0, top)
        a = x - low
        e = np.exp(a)
        s = e.sum(1, keepdims=True)
        p = np.divide(e, s, out=np.zeros_like(e), where=s != 0)
        return p, (low + np.log(s))[:, 0], np.where(np.isneginf(top), 0.0, a)


def gate_ref(x, m, live=None, normalised=False):
    x = x.copy()
    if live is not None:
        x[~live] = -np.inf
    N, K = x.shape
    ids = np.full((N, m), -1, dtype=np.int64)
    order = np.argsort(-x, axis=1, kind="stable")[:, :m]
    ids[:, :order.shape[1]] = np.where(np.isneginf(np.take_along_axis(x, order, 1)), -1, order)
    p, lse, a = softmax_ref(x)
    gamma = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0.0)
    if normalised:
        s = gamma.sum(1, keepdims=True)
        gamma = np.divide(gamma, s, out=np.zeros_like(gamma), where=s != 0)
    return ids, gamma, lse, p, a


def balance_ref(ids, p, rows):
    K = p.shape[1]
    counts = np.bincount(ids[ids >= 0], minlength=K)
    mass, total = p.sum(0), counts.sum() * rows
    share = K * counts / total if total else np.zeros(K)
    return counts, mass, share, float((share * mass).sum())


def gate_grad_ref(p, ids, gamma, dgamma, share, coef, normalised):
    v = np.where(ids >= 0, gamma * dgamma, 0.0)
    S = v.sum(1, keepdims=True)
    if normalised:
        v = v - np.where(ids >= 0, gamma, 0.0) * S
        S = np.zeros_like(S)
    d = -p * S
    if share is not None:
        d = d + coef * p * (share - (p * share).sum(1, keepdims=True))
    for t in range(ids.shape[1]):
        r = np.nonzero(ids[:, t] >= 0)[0]
        d[r, ids[r, t]] += v[r, t]
    return d


def distill_ref(x, ids, values, kind, T, w, scale):
    """rows, loss, dL; and q, u (the teacher's exponents), for bounds."""
    N, K = x.shape
    ok = (ids >= 0) & (ids < K)
    with np.errstate(all="ignore"):
        u = np.where(ok, (np.log(values) if kind == "gamma" else values) / T, -np.inf)
        q, _, b = softmax_ref(u)
        p, lse, _ = softmax_ref(x / T)
        at = np.where(ok, ids, 0)
        logp = np.take_along_axis(x / T, at, 1) - lse[:, None]
        logq = b - np.log(np.exp(b).sum(1, keepdims=True))
        kl = np.where(q > 0, q * (logq - logp), 0.0).sum(1)
    kl[np.isneginf(x).all(1)] = np.inf
    on = (w != 0) & np.isfinite(u).any(1)
    rows = np.where(on, w * T * T * np.where(on, kl, 0.0), 0.0)
    d = p.copy()
    for t in range(ids.shape[1]):
        r = np.nonzero(ok[:, t])[0]
        d[r, ids[r, t]] -= q[r, t]
    d *= np.where(on, w, 0.0)[:, None] * scale * T
    return rows, scale * rows.sum(), d, p, q, u, on


def test_restatements_by_hand():
    x = np.log(np.array([[1.0, 2, 5], [4, 4, 2]]))
    ids, gamma, lse, p, _ = gate_ref(x, 2)
    assert ids.tolist() == [[2, 1], [0, 1]]
    assert np.allclose(gamma, [[5 / 8, 2 / 8], [0.4, 0.4]]) and np.allclose(lse, np.log([8, 10]))
    counts, mass, share, loss = balance_ref(ids, p, 2)
    assert counts.tolist() == [1, 2, 1] and np.allclose(mass, [1 / 8 + 0.4, 1 / 4 + 0.4, 5 / 8 + 0.2])
    assert np.allclose(share, 3 * np.array([1, 2, 1]) / 8) and np.isclose(loss, 3 / 8 * (2 + 0.65))
    rows, loss, d, *_ = distill_ref(x[:1], np.array([[2, 0]]), np.array([[0.75, 0.25]]), "gamma", 1.0,
                                    np.ones(1), 1.0)
    assert np.isclose(loss, 0.75 * np.log(0.75 * 8 / 5) + 0.25 * np.log(0.25 * 8))
    assert np.allclose(d, [[1 / 8 - 0.25, 1 / 4, 5 / 8 - 0.75]])


@pytest.mark.parametrize("normalised", [False, True])
def test_gate_gradient_against_differences(normalised):
    rng = np.random.default_rng(3)
    x, c = rng.standard_normal((4, 7)), rng.standard_normal((4, 3))
    ids, gamma, _, p, _ = gate_ref(x, 3, normalised=normalised)
    share = balance_ref(ids, p, 4)[2]

    def loss(x):
        _, gam, _, p, _ = gate_ref(x, 3, normalised=normalised)
        return (c * gam).sum() + 0.7 * (share * p.sum(0)).sum()

    d = gate_grad_ref(p, ids, gamma, c, share, 0.7, normalised)
    _differences(loss, x, d)


@pytest.mark.parametrize("kind,T", [("gamma", 1.0), ("logits", 2.0), ("gamma", 0.5)])
def test_distill_gradient_against_differences(kind, T):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 6))
    ids, v, w = np.array([[1, 4, -1], [5, 0, 2], [3, 3, 1]]), rng.random((3, 3)), np.array([1.0, 0.5, 2])
    d = distill_ref(x, ids, v, kind, T, w, 0.3)[2]
    _differences(lambda x: distill_ref(x, ids, v, kind, T, w, 0.3)[1], x, d)


def _differences(loss, x, d, h=1e-5):
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        assert abs((loss(a) - loss(b)) / (2 * h) - d[i]) < 1e-7, i


# --------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from soft_clustering_gb300 import build
    build.build()
    return G.lib()


def test_sizes(lib):
    assert G.gmm_gate_ws_bytes(1000, 64, 2) > 0 and G.gmm_gate_ws_bytes(0, 1, 1) > 0
    for bad in ((-1, 64, 2), (10, 0, 2), (10, 65537, 2), (10, 64, 0), (10, 64, 9), (2 ** 30, 64, 4)):
        assert G.gmm_gate_ws_bytes(*bad) == 0, bad
    assert G.gmm_distill_ws_bytes() > 0


def test_refusals_before_anything_is_queued(lib):
    bad, P, big = G.GMM_ERR_INVALID_ARG, 4096, 1 << 40

    def each(f, args, wrong):
        for i, v in wrong:
            a = list(args)
            a[i] = v
            assert f(*a) == bad, (f.__name__, i, v)

    gate = [P, 1, 10, 64, 2, 0, P, P, P, P, P, P, P, P, P, big, None]
    each(lib.gmm_gate, gate, [(0, None), (0, P + 1), (1, 3), (1, -1), (2, -1), (2, 2 ** 31), (3, 0), (3, 65537),
                              (4, 0), (4, 9), (5, 2), (7, None), (7, P + 2), (8, None), (8, P + 1), (9, P + 2),
                              (10, None), (10, P + 4), (11, None), (11, P + 2), (12, None), (12, P + 1),
                              (13, None), (13, P + 2), (14, None), (14, P + 128)])
    gate[15] = G.gmm_gate_ws_bytes(10, 64, 2) - 1
    assert lib.gmm_gate(*gate) == G.GMM_ERR_WORKSPACE
    grad = [P, 1, 10, 64, 2, 0, P, P, P, P, P, 0.5, P, None]
    each(lib.gmm_gate_grad, grad, [(0, None), (0, P + 1), (1, 3), (2, -1), (3, 0), (3, 65537), (4, 0), (4, 9),
                                   (5, 4), (7, None), (7, P + 1), (8, None), (8, P + 2), (9, P + 2), (10, P + 1),
                                   (12, None), (12, P + 1)])
    dist = [P, 1, 10, 64, 2, 0, 0, 1.0, 1.0, P, P, P, P, P, P, P, big, None]
    each(lib.gmm_distill, dist, [(0, None), (0, P + 1), (1, 3), (2, -1), (3, 0), (3, 2 ** 18 + 1), (4, 0), (4, 65),
                                 (5, 2), (6, 2), (7, 0.0), (7, -1.0), (7, float("nan")), (7, float("inf")),
                                 (7, 1e-300), (9, None), (9, P + 2), (10, None), (10, P + 1), (11, P + 2),
                                 (12, None), (12, P + 2), (13, None), (13, P + 1), (14, P + 1), (15, None),
                                 (15, P + 128)])
    dist[16] = G.gmm_distill_ws_bytes() - 1
    assert lib.gmm_distill(*dist) == G.GMM_ERR_WORKSPACE


def test_no_rows_is_no_work(lib):
    assert lib.gmm_gate(None, 0, 0, 8, 2, 0, None, None, None, None, None, None, None, None, None, 0, None) == G.GMM_OK
    assert lib.gmm_gate_grad(None, 0, 0, 8, 2, 0, None, None, None, None, None, 0.0, None, None) == G.GMM_OK


def test_python_refusals(monkeypatch):
    import torch
    from soft_clustering_gb300 import gate
    for make in (lambda: gate.Gate(4, 8, 2, torch.float16, device="cpu"),
                 lambda: gate.Distiller(4, 8, 2, torch.float16, device="cpu")):
        with pytest.raises(ValueError, match="CUDA device"):
            make()
    for make in (lambda: gate.Gate(4, 8, 9, torch.float16), lambda: gate.Gate(4, 0, 1, torch.float16),
                 lambda: gate.Gate(4, 8, 2, torch.float64), lambda: gate.Distiller(4, 8, 65, torch.float32),
                 lambda: gate.Distiller(4, 2 ** 18 + 1, 2, torch.float32),
                 lambda: gate.Distiller(4, 8, 2, torch.float32, teacher="ids"),
                 lambda: gate.Distiller(4, 8, 2, torch.float32, temperature=0.0),
                 lambda: gate.Distiller(4, 8, 2, torch.float32, temperature=float("nan")),
                 lambda: gate.Distiller(2 ** 30, 8, 4, torch.float32)):
        with pytest.raises(ValueError):
            make()
    # every call looks at the device, the shapes and what went before
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    there = torch.device("cuda", 1)
    x, c = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4, 2)
    g, d = object.__new__(gate.Gate), object.__new__(gate.Distiller)
    for o in (g, d):
        o.N, o.K, o.m, o.dtype, o.xdtype, o.device = 4, 8, 2, torch.float16, 1, torch.device("cpu")
        o._shape, o._small = (4, 8), (4, 2)
    g._balanced, g.flags = None, 0
    with pytest.raises(RuntimeError, match="before forward"):
        g.backward(x, c)
    g._balanced = False
    with pytest.raises(RuntimeError, match="no balance"):
        g.backward(x, c, balance=0.1)
    for call in (lambda: g.forward(x.float()), lambda: g.forward(x[:3]), lambda: g.forward(x.T.contiguous().T),
                 lambda: g.forward(x, live=torch.ones(4)), lambda: g.forward(x, live=torch.ones(3, dtype=torch.bool)),
                 lambda: g.backward(x, c.half()), lambda: g.backward(x, c[:, :1]), lambda: g.backward(x, c, out=x[:2]),
                 lambda: d.loss(x, c, c), lambda: d.loss(x, c.int(), c.half()), lambda: d.loss(x, c.int(), c, weights=c),
                 lambda: d.step(x, c.int(), c, add=True), lambda: d.step(x, c.int(), c, out=x.float())):
        with pytest.raises(ValueError):
            call()
    monkeypatch.setattr(gate, "_need", lambda t, *a: t)
    monkeypatch.setattr(gate, "_empty", lambda *a: x)
    g.device = d.device = there
    for call in (lambda: g.forward(x), lambda: g.backward(x, c), lambda: d.loss(x, c.int(), c),
                 lambda: d.step(x, c.int(), c)):
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


def _f64(t):
    return t.detach().double().cpu().numpy()


def _logits(rng, N, K, dtype, plain=False):
    """Logits as the type holds them, with the rows that go wrong first."""
    import torch
    x = rng.standard_normal((N, K)).astype(np.float32) * 2
    if not plain:
        if N > 8:
            x[0] = -np.inf                       # nothing left
            x[1] = -np.inf
            x[1, K // 2] = 3.0                   # one left
            x[2] = 0.5                           # all the same
            x[3] = float(torch.finfo(_dt(dtype)).min)
            x[4] = np.where(rng.random(K) < 0.5, -0.0, 0.0)
            x[5] = float(torch.finfo(_dt(dtype)).min)
            x[5, K - 1] = 1.0
            x[6] = np.where(rng.random(K) < 0.7, -np.inf, x[6])
            x[7] = x[7] * 20 - 60                # far below zero, sharp
        x[N // 2:] = np.round(x[N // 2:] * 4) / 4  # ties
    return torch.from_numpy(x).to(_dt(dtype)).cuda()


def _misaligned(t):
    """The same values one element past an aligned address."""
    import torch
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    room.copy_(t.reshape(-1))
    return room.view(t.shape)


def _E(a):
    with np.errstate(invalid="ignore"):
        return np.where(np.isfinite(a), 4 * U * np.abs(a) + 2.0 ** -21, 0.0)


def _S(p, a):
    return 300 * U + np.nansum(p * _E(a), 1, keepdims=True)


def _near(got, ref, bound, what):
    got = _f64(got) if not isinstance(got, np.ndarray) else got
    assert got.shape == ref.shape, what
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), what
    off = np.where(fine, np.abs(np.where(fine, got, 0.0) - np.where(fine, ref, 0.0)) - bound, -1.0)
    assert (off <= 0).all(), (what, off.max(), np.unravel_index(off.argmax(), off.shape))


# K around each form's borders; N odd, and more rows than blocks
SIZES = [(1, 1, 1), (9, 1, 2), (10, 2, 8), (33, 3, 2), (700, 7, 3), (1200, 8, 2), (65, 9, 4), (129, 16, 1),
         (77, 31, 3), (500, 33, 2), (2049, 64, 2), (64, 65, 8), (99, 100, 5), (150, 127, 2), (41, 255, 4),
         (640, 256, 4), (70, 257, 8), (21, 1000, 2), (900, 1024, 2), (35, 1025, 3), (12, 2048, 8), (17, 2500, 4),
         (400, 4096, 4), (13, 4097, 1), (11, 8192, 2), (9, 10007, 3), (10, 16384, 4), (12, 16392, 2), (3, 32768, 8),
         (9, 33333, 4), (9, 65535, 2), (10, 65536, 4), (1, 65536, 8), (2, 50000, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,K,m", SIZES)
def test_gate(cuda, N, K, m, dtype):
    import torch
    from soft_clustering_gb300.gate import Gate
    rng = np.random.default_rng(N * 31 + K)
    for case in range(4):
        normalised, shifted, padded, balance = case & 1, case >= 2, case in (1, 2), case != 2
        L = _logits(rng, N, K, dtype)
        if shifted:
            L = _misaligned(L)
        x = _f64(L)
        live = rng.random(N) < 0.8 if padded else None
        if padded:
            L[torch.from_numpy(~live).cuda()] = float("nan")  # padding is not read
        dlive = torch.from_numpy(live).cuda() if padded else None
        g = Gate(N, K, m, L.dtype, normalised=bool(normalised))
        ids, gamma = g.forward(L, live=dlive, balance=balance)
        rid, rg, rl, p, a = gate_ref(x, m, live, normalised)
        assert np.array_equal(ids.cpu().numpy(), rid), (case, "ids")
        S, E = _S(p, a), _E(a)
        at = np.maximum(rid, 0)
        rel = np.take_along_axis(E, at, 1) + S + 4 * U
        if normalised:
            rel = rel + (rg * rel).sum(1, keepdims=True) + 8 * U
        _near(gamma, rg, rg * rel + 2.0 ** -120, "gamma")
        fine = np.where(np.isfinite(rl), rl, 0.0)
        logs = np.log(np.maximum(1.0, np.exp(a).sum(1)))
        _near(g.lse, rl, S[:, 0] + 4 * U * (np.abs(fine) + logs) + 4 * U, "lse")
        share = None
        relp = E + S + 4 * U
        if balance:
            rows = int((np.isfinite(rl)).sum())
            rc, rm, share, loss = balance_ref(rid, p, rows)
            assert np.array_equal(g.counts.cpu().numpy(), rc)
            bm = (p * relp).sum(0) + (N / 100 + 64) * U * rm + N * 2.0 ** -120
            _near(g.mass, rm, bm, "mass")
            _near(g.share, share, 2 * U * share, "share")
            _near(_f64(g.loss), np.array([loss]), (share * (bm + 4 * U * rm)).sum() + 2 * U * loss, "loss")
        # the gradient, from the gate's own ids, gamma and share
        dg = torch.from_numpy(rng.standard_normal((N, m)).astype(np.float32)).cuda()
        kg, kd = _f64(gamma), np.where(rid >= 0, _f64(dg), 0.0)
        dg[torch.from_numpy(rid < 0).cuda()] = float("nan")  # of entries left out
        coef = 0.3 if balance else 0.0
        sh = _f64(g.share) if balance else None
        for d_gamma in (dg, None):
            if d_gamma is None:
                kd = np.zeros_like(kd)
            out = torch.full_like(L, 7.0)
            if shifted:
                out = _misaligned(out)
            got = g.backward(L, d_gamma, live=dlive, balance=coef, out=out)
            ref = gate_grad_ref(p, rid, kg, kd, sh, coef, normalised)
            v = np.abs(kg * kd)
            if normalised:
                v = v + kg * v.sum(1, keepdims=True)
            per = v.sum(1, keepdims=True) + np.zeros((1, K))
            if balance:
                per = per + coef * (sh + (p * sh).sum(1, keepdims=True))
            size = p * per
            for t in range(m):
                r = np.nonzero(rid[:, t] >= 0)[0]
                size[r, rid[r, t]] += v[r, t]
            # an exponential e below 2^-126 may be 0 (above), and the gradient is e / sum times at most `per`, with
            # sum >= 1: 2^-126 per more
            _near(got, ref, (relp + 2 * S + 340 * U) * size + UT[dtype] * np.abs(ref) + SUB[dtype] + 2.0 ** -126 * per,
                  "dlogits")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,K", [("f32", 9000), ("bf16", 9001), ("f16", 16385), ("bf16", 16392), ("f16", 2048),
                                     ("f32", 1025), ("bf16", 520), ("f16", 24)])
def test_balance_of_many_rows(cuda, K, dtype):
    """More rows than blocks keep sums for, in every form: rows, entries and mass of all of them."""
    from soft_clustering_gb300.gate import Gate
    N, m = 1300 if K < 5000 else 330, 2
    L = _logits(np.random.default_rng(K), N, K, dtype, plain=True)
    g = Gate(N, K, m, L.dtype)
    ids, _ = g.forward(L, balance=True)
    rid, _, rl, p, a = gate_ref(_f64(L), m)
    assert np.array_equal(ids.cpu().numpy(), rid)
    rc, rm, share, loss = balance_ref(rid, p, N)
    assert np.array_equal(g.counts.cpu().numpy(), rc)
    bm = (p * (_E(a) + _S(p, a) + 4 * U)).sum(0) + (N / 100 + 64) * U * rm + N * 2.0 ** -120
    _near(g.mass, rm, bm, "mass")
    _near(g.share, share, 2 * U * share, "share")
    _near(g.loss, np.array([loss]), (share * (bm + 4 * U * rm)).sum() + 2 * U * loss, "loss")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [5, 64, 200, 1024, 3001, 20000])
def test_gate_of_rows_that_are_not_finite(cuda, K, dtype):
    """A NaN is the largest; it and +inf show in gamma and lse of their row, and in no other."""
    import torch
    from soft_clustering_gb300.gate import Gate
    rng = np.random.default_rng(K)
    L = _logits(rng, 12, K, dtype, plain=True)
    want_ids, want_gamma = [t.clone() for t in Gate(12, K, 2, L.dtype).forward(L)]
    L[3, K - 1], L[5, K // 2], L[7] = float("nan"), float("inf"), float("nan")
    neg = torch.tensor([-1], dtype=torch.int16 if dtype != "f32" else torch.int32, device="cuda").view(L.dtype)
    L[9, 1] = neg[0]  # a NaN with its sign set
    g = Gate(12, K, 2, L.dtype)
    ids, gamma = g.forward(L)
    odd = [3, 5, 7, 9]
    even = [n for n in range(12) if n not in odd]
    assert ids[odd, 0].tolist() == [K - 1, K // 2, 0, 1] and int(ids[7, 1]) == 1
    assert torch.isnan(gamma[odd]).all() and torch.isnan(g.lse[odd]).all()
    assert torch.equal(ids[even], want_ids[even]) and torch.equal(gamma[even], want_gamma[even])
    assert torch.isfinite(g.lse[even]).all()
    d = g.backward(L, torch.ones(12, 2, device="cuda"))
    assert torch.isnan(d[odd]).all() and torch.isfinite(d[even]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [6, 64, 300, 1024, 5000, 40000])
def test_gate_gradient_of_entries_that_are_not_the_gates(cuda, K, dtype):
    """An id twice, ids outside [0, K): through the C ABI."""
    import torch
    rng = np.random.default_rng(K)
    N, m = 20, 4
    L = _logits(rng, N, K, dtype, plain=True)
    ids = rng.integers(0, K, (N, m)).astype(np.int32)
    ids[:5, 2] = ids[:5, 0]
    ids[3] = ids[3, 0]
    ids[6, 1], ids[7, 0], ids[8, 3] = -1, K, 2 ** 31 - 1
    gam, dg = rng.random((N, m)).astype(np.float32), rng.standard_normal((N, m)).astype(np.float32)
    known = np.where(ids < K, ids, -1)
    p, _, a = softmax_ref(_f64(L))
    relp = _E(a) + 3 * _S(p, a) + 340 * U
    for normalised in (0, 1):
        out = torch.empty_like(L)
        G.gmm_gate_grad(L, CODE[dtype], N, K, m, normalised, None, torch.from_numpy(ids).cuda(),
                        torch.from_numpy(gam).cuda(), torch.from_numpy(dg).cuda(), None, 0.0, out)
        ref = gate_grad_ref(p, known, gam.astype(float), dg.astype(float), None, 0.0, normalised)
        v = np.where(known >= 0, np.abs(gam * dg), 0.0).astype(float)
        v = v + np.where(known >= 0, gam, 0.0) * v.sum(1, keepdims=True) * normalised
        size = p * v.sum(1, keepdims=True)
        for t in range(m):
            r = np.nonzero(known[:, t] >= 0)[0]
            size[r, known[r, t]] += v[r, t]
        _near(out, ref, relp * size + UT[dtype] * np.abs(ref) + SUB[dtype], "dlogits")


DISTILL = [(1, 1, 1), (10, 2, 2), (700, 7, 3), (1300, 8, 4), (33, 31, 5), (900, 64, 4), (20, 65, 33), (11, 100, 64),
           (300, 256, 4), (77, 257, 8), (50, 1000, 16), (400, 1024, 2), (30, 1025, 9), (12, 4096, 32), (700, 4096, 3),
           (9, 10007, 5), (11, 16384, 64), (10, 16385, 7), (9, 50257, 32), (3, 65536, 64), (200, 65536, 2), (9, 70001, 3),
           (10, 131072, 64), (1, 131071, 1), (9, 200001, 10), (2, 262144, 64), (10, 262143, 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,K,m", DISTILL)
def test_distill(cuda, N, K, m, dtype):
    import torch
    from soft_clustering_gb300.gate import Distiller
    rng = np.random.default_rng(N * 17 + K)
    for kind, T, weighted, shifted in (("gamma", 1.0, False, False), ("logits", 2.0, True, True),
                                       ("gamma", 0.5, True, False)):
        L = _logits(rng, N, K, dtype)
        if N > 8:
            L[3] = L[5] = 0.0  # losses past fp32 are another test's
        x = _f64(L)
        ids = rng.integers(0, K, (N, m)).astype(np.int32)  # some of them twice
        vals = (rng.standard_normal((N, m)) * 3).astype(np.float32)
        if kind == "gamma":
            vals = np.exp(vals - 4).astype(np.float32)
        if N > 8:
            ids[1, 0] = K // 2                       # the one component that row 1 has
            if m > 1:
                ids[1, 1:] = -1
            ids[2] = -1                              # no entry
            ids[7, 0], vals[6, m - 1] = K, 0.0 if kind == "gamma" else -np.inf
        w = rng.random(N).astype(np.float32) + 0.5 if weighted else np.ones(N, dtype=np.float32)
        if weighted and N > 8:
            w[N - 1] = 0.0
            L[N - 1] = float("nan")                  # padding is not read
        scale = 0.25
        ref, loss, rd, p, q, u, on = distill_ref(x, ids, vals.astype(float), kind, T, w.astype(float), scale)
        if shifted:
            L = _misaligned(L)
        d = Distiller(N, K, m, L.dtype, teacher=kind, temperature=T, scale=scale)
        args = L, torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda()
        dw = torch.from_numpy(w).cuda() if weighted else None
        # bounds
        _, _, a = softmax_ref(x / T)
        S = _S(p, a)
        ok = np.isfinite(u)
        with np.errstate(all="ignore"):
            umax = np.where(ok, np.abs(u), 0.0).max(1, keepdims=True)
            spread = np.where(ok, np.abs(u - np.where(ok, u, -np.inf).max(1, keepdims=True)), 0.0)
            relq = 16 * U * umax + 4 * U * spread + 2.0 ** -20 + 300 * U
            at = np.where((ids >= 0) & (ids < K), ids, 0)
            la = np.where(ok & (q > 0), np.abs(np.take_along_axis(a, at, 1)), 0.0)
            la = np.where(np.isfinite(la), la, 0.0)
            size = 1 + umax[:, 0] + (q * (spread + la)).sum(1) + np.log(np.maximum(1, np.exp(a).sum(1)))
        br = w * T * T * ((relq * q).sum(1) + S[:, 0] + 64 * U) * size
        total = d.loss(*args, weights=dw)
        _near(d.rows, ref, br, "rows")
        if np.isfinite(loss):
            _near(total, np.array([loss]), scale * br.sum() + 2 * U * abs(loss), "loss")
        else:
            assert float(total) == loss
        rows = d.rows.clone()
        relp = _E(a) + S + 4 * U
        big = np.abs(scale * w * T)[:, None] * p * relp
        peak = np.abs(scale * w * T)[:, None] * q * (relq + 8 * U)
        for t in range(m):
            r = np.nonzero((ids[:, t] >= 0) & (ids[:, t] < K))[0]
            big[r, ids[r, t]] += peak[r, t]
        full = 8 * U * np.abs(scale * w * T)[:, None] * p
        got_total, got = d.step(*args, weights=dw, out=_misaligned(torch.full_like(L, 5.0)) if shifted else None)
        assert torch.equal(d.rows, rows)
        _near(got, rd, big + full + UT[dtype] * np.abs(rd) + SUB[dtype] + 4 * U * np.abs(rd), "dlogits")
        # added to what is there
        base = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).to(L.dtype).cuda()
        if shifted:
            base = _misaligned(base)
        want = _f64(base) + rd
        d.step(*args, weights=dw, out=base, add=True)
        _near(base, want, big + full + (UT[dtype] + 2 * U) * np.abs(want) + SUB[dtype] + 4 * U * np.abs(rd), "added")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [6, 64, 300, 1024, 5000, 40000])
def test_distill_of_what_is_not_there(cuda, K, dtype):
    """A student with -inf where the teacher has a share; logits that T takes past
    fp32; NaN in one row alone."""
    import torch
    from soft_clustering_gb300.gate import Distiller
    rng = np.random.default_rng(K)
    N, m = 10, 2
    L = _logits(rng, N, K, dtype, plain=True)
    ids = np.stack([np.zeros(N), np.full(N, K - 1)], 1).astype(np.int32)
    vals = np.full((N, m), 0.5, dtype=np.float32)
    L[1] = float("-inf")                 # nothing
    L[2, 0] = float("-inf")              # not the teacher's first
    L[3, K // 2] = float("nan")
    L[4] = float(torch.finfo(L.dtype).min)
    L[4, 0] = L[4, K - 1] = 1.0
    vals[5, 1] = float("nan")
    d = Distiller(N, K, m, L.dtype, temperature=0.5)
    total, got = d.step(L, torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda())
    rows = _f64(d.rows)
    assert rows[1] == rows[2] == np.inf and np.isnan(rows[3]) and np.isnan(rows[5])
    assert np.isnan(float(total))
    fine = [0, 4, 6, 7, 8, 9]
    assert np.isfinite(rows[fine]).all() and np.isfinite(_f64(got)[fine + [1, 2]]).all()
    assert np.isnan(_f64(got)[3]).all()
    ref = np.zeros(K)
    ref[[0, K - 1]] = -0.5 * 0.5 / N
    _near(got[1], ref, UT[dtype] * np.abs(ref) + SUB[dtype] + 2.0 ** -18 * np.abs(ref), "no student")
    assert abs(rows[4]) < 1e-6  # both have one half


@pytest.mark.gpu
def test_no_rows(cuda):
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    L = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    g = Gate(0, 16, 2, L.dtype)
    ids, gamma = g.forward(L, balance=True)
    assert ids.shape == gamma.shape == (0, 2)
    assert not g.counts.any() and not g.mass.any() and not g.share.any() and float(g.loss) == 0.0
    assert g.backward(L, gamma, balance=1.0).shape == (0, 16)
    d = Distiller(0, 16, 2, L.dtype)
    total, out = d.step(L, ids, gamma)
    assert float(total) == 0.0 and out.shape == (0, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(5000, 64), (3000, 256), (2000, 1000), (700, 4096), (40, 40001)])
def test_results_repeat_to_the_bit(cuda, N, K):
    import torch
    from soft_clustering_gb300.gate import Distiller, Gate
    rng = np.random.default_rng(N)
    L = _logits(rng, N, K, "bf16")
    g, d = Gate(N, K, 2, L.dtype), Distiller(N, K, 2, L.dtype)
    first = None
    for _ in range(3):
        ids, gamma = g.forward(L, balance=True)
        out = [t.clone() for t in (ids, gamma, g.lse, g.counts, g.mass, g.share, g.loss)]
        out.append(g.backward(L, gamma, balance=0.1))
        total, grad = d.step(L, ids, gamma)
        out += [total.clone(), grad, d.rows.clone()]
        first = first or out
        for a, b in zip(first, out):
            assert torch.equal(a, b) or (a.isnan() == b.isnan()).all()
