"""Local experts behind the soft assignment (gmm_route, gmm_spread,
gmm_collect, gmm_expert_product and its gradients, LocalExperts).

CPU: refusals, sizes, and the 64-bit restatements against a hand-worked
example.  GPU: the kernels against the restatements.

Tolerances, from the operations alone (u = 2^-24, uT the unit roundoff of the
type: 0 for fp32, 2^-11 for fp16, 2^-8 for bf16; fp16 results below 2^-14
also lose up to 2^-25):
  route    equality
  spread   (u + uT) |y|;  dgamma: (D + 1) u sum |x z|
  collect  (m + 1) u sum |w z| + uT |out|
  product  2 L u sum |p q| + uT |y| over a contraction of L terms (each step
           of a tensor core's running sum may be cut off, not rounded)
Products of small whole numbers are exact in fp32 and have to be equal.
"""
import ctypes

import numpy as np
import pytest

import soft_clustering_gb300 as G

U = 2.0 ** -24
UT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
CODE = {"f32": G.GMM_F32, "f16": G.GMM_F16, "bf16": G.GMM_BF16}


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


# ------------------------------------------------------- restatements, 64 bits

def route_ref(ids, K):
    flat = np.asarray(ids).reshape(-1)
    lists = [[] for _ in range(K)]
    for e, k in enumerate(flat):
        if 0 <= k < K:
            lists[k].append(e)
    offsets = np.zeros(K + 1, dtype=np.int64)
    offsets[1:] = np.cumsum([len(x) for x in lists])
    entry = np.full(flat.size, -1, dtype=np.int32)
    slot = np.full(flat.size, -1, dtype=np.int32)
    for k in range(K):
        for i, e in enumerate(lists[k]):
            entry[offsets[k] + i] = e
            slot[e] = offsets[k] + i
    return offsets, entry, slot.reshape(np.asarray(ids).shape)


def product_ref(A, W, offsets):
    Y = np.zeros((A.shape[0], W.shape[1]))
    for k in range(W.shape[0]):
        a, b = offsets[k], offsets[k + 1]
        Y[a:b] = A[a:b] @ W[k].T
    return Y


def dw_ref(dY, A, offsets, K):
    dW = np.zeros((K, dY.shape[1], A.shape[1]))
    for k in range(K):
        a, b = offsets[k], offsets[k + 1]
        dW[k] = dY[a:b].T @ A[a:b]
    return dW


def test_restatement_by_hand():
    ids = np.array([[2, 0], [0, -1], [3, 2]], dtype=np.int32)  # K = 3: id 3 is left out
    o, e, s = route_ref(ids, 3)
    assert o.tolist() == [0, 2, 2, 4]
    assert e.tolist() == [1, 2, 0, 5, -1, -1]
    assert s.tolist() == [[2, 0], [1, -1], [-1, 3]]
    A = np.array([[1.0, 2], [3, 4], [5, 6], [7, 8], [9, 9], [9, 9]])
    W = np.array([[[1.0, 1]], [[5, 5]], [[2, -1]]])
    assert product_ref(A, W, o).reshape(-1).tolist() == [3, 7, 4, 6, 0, 0]
    assert dw_ref(np.ones((6, 1)), A, o, 3).reshape(3, 2).tolist() == [[4, 6], [0, 0], [12, 14]]


# --------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from soft_clustering_gb300 import build
    build.build()
    return G.lib()


def test_sizes(lib):
    assert G.gmm_route_ws_bytes(1000, 4, 64) > 0
    assert G.gmm_route_ws_bytes(0, 4, 64) > 0
    for bad in ((-1, 4, 64), (10, 0, 64), (10, 9, 64), (10, 4, 0), (10, 4, 65537), (2 ** 30, 4, 4)):
        assert G.gmm_route_ws_bytes(*bad) == 0, bad
    assert G.gmm_expert_ws_bytes(0, 128, 128, 8, G.GMM_F16) > 0
    for bad in ((-1, 8, 8, 1, 0), (1, 0, 8, 1, 0), (1, 8, 0, 1, 0), (1, 8, 8, 0, 0),
                (1, 8, 8, 70000, 0), (1, 65536, 65536, 1, 0), (1, 8, 8, 1, 3), (2 ** 31, 8, 8, 1, 0)):
        assert G.gmm_expert_ws_bytes(*bad) == 0, bad


def test_refusals_before_anything_is_queued(lib):
    bad, P = G.GMM_ERR_INVALID_ARG, 256
    big = 1 << 40
    assert lib.gmm_route(P, 10, 2, 4, None, P, P, P, big, None) == bad
    assert lib.gmm_route(None, 10, 2, 4, P, P, P, P, big, None) == bad
    assert lib.gmm_route(P, 10, 9, 4, P, P, P, P, big, None) == bad
    assert lib.gmm_route(P, 10, 2, 4, P, P, P, P, 0, None) == G.GMM_ERR_WORKSPACE
    for x, N, D, m, K, R in ((7, 1, 8, 1, 1, 1), (0, -1, 8, 1, 1, 1), (0, 1, 0, 1, 1, 1),
                             (0, 1, 8, 0, 1, 1), (0, 1, 8, 9, 1, 1), (0, 1, 8, 1, 0, 1),
                             (0, 1, 8, 1, 1, -1)):
        assert lib.gmm_spread(P, x, N, D, m, K, R, P, P, None, None, P, None, None) == bad
    assert lib.gmm_spread(None, 0, 1, 8, 1, 1, 1, P, P, None, None, P, None, None) == bad
    assert lib.gmm_spread(P, 0, 1, 8, 1, 1, 1, P, P, None, P, P, None, None) == bad  # Z alone
    assert lib.gmm_spread(P, 0, 1, 8, 1, 1, 1, P, P, None, None, P, P, None) == bad  # dgamma alone
    assert lib.gmm_spread(P + 1, 1, 1, 8, 1, 1, 1, P, P, None, None, P, None, None) == bad
    assert lib.gmm_collect(P, 0, 1, 8, 1, 1, None, None, P, None) == bad
    assert lib.gmm_collect(P, 0, 1, 8, 1, 1, P, None, P + 2, None) == bad
    ok = lib.gmm_expert_ws_bytes(4, 8, 8, 2, 1)
    for f in (lib.gmm_expert_product, lib.gmm_expert_product_dx):
        assert f(P, 1, 4, 8, 8, 2, P, P, P, P, ok - 1, None) == G.GMM_ERR_WORKSPACE
        assert f(P, 1, 4, 8, 8, 2, None, P, P, P, ok, None) == bad
        assert f(None, 1, 4, 8, 8, 2, P, P, P, P, ok, None) == bad
        assert f(P, 5, 4, 8, 8, 2, P, P, P, P, ok, None) == bad
        assert f(P, 1, 4, 8, 8, 2, P, P, P, P + 8, ok, None) == bad  # workspace alignment
        assert f(P + 1, 1, 4, 8, 8, 2, P, P, P, P, ok, None) == bad
    assert lib.gmm_expert_product_dw(P, P, 1, 4, 8, 8, 2, P, P, 2, P, ok, None) == bad  # bf16 of f16


def test_no_points_is_no_work(lib):
    assert lib.gmm_spread(None, 0, 0, 8, 2, 4, 0, None, 256, None, None, None, None, None) == G.GMM_OK
    assert lib.gmm_collect(None, 0, 0, 8, 2, 0, None, None, None, None) == G.GMM_OK


def test_header_says_what_the_binding_passes():
    assert ctypes.sizeof(G.gmm_adamw_tensor) == 8 * 8 + 8
    assert ctypes.sizeof(G.gmm_adamw_opts) == 6 * 8 + 8 + 8 + 8


# -------------------------------------------------------------------------- GPU

@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def _ids(rng, N, m, K, drop):
    ids = np.full((N, m), -1, dtype=np.int32)
    first = rng.integers(0, K, N)
    for t in range(m):
        ids[:, t] = (first + t * max(1, K // m)) % K if t < K else -1
    ids[rng.random((N, m)) < drop] = -1
    if N > 3:
        ids[1] = -1            # a point with nothing left
        ids[2, 0] = K          # just past the last component
        ids[3, 0] = -2 ** 31
    return ids


def _rand(rng, shape, dtype, whole=False):
    import torch
    x = rng.integers(-2, 3, shape).astype(np.float32) if whole else rng.standard_normal(shape).astype(np.float32)
    return torch.from_numpy(x).to(_dt(dtype)).cuda()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _near(got, ref, bound, what):
    got = _f64(got)
    assert got.shape == ref.shape, what
    off = np.abs(got - ref) - bound
    assert np.isfinite(got).all() and (off <= 0).all(), (what, off.max(), np.unravel_index(off.argmax(), off.shape))


ROUTES = [(0, 2, 5, 0.0), (1, 1, 1, 0.0), (1, 8, 4096, 0.0), (5, 4, 3, 0.3), (256, 4, 64, 0.1),
          (257, 4, 64, 0.1), (1500, 1, 7, 0.0), (5000, 8, 300, 0.5), (20011, 3, 4096, 0.2),
          (40000, 2, 65536, 0.1), (3000, 2, 20000, 1.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("N,m,K,drop", ROUTES)
def test_route(cuda, N, m, K, drop):
    import torch
    from soft_clustering_gb300.experts import Router
    rng = np.random.default_rng(N + 7 * m + K)
    ids = _ids(rng, N, m, K, drop)
    r = Router(N, m, K)
    for _ in range(2):  # the second call finds its own outputs and workspace
        r.route(torch.from_numpy(ids).cuda())
    o, e, s = route_ref(ids, K)
    assert np.array_equal(r.offsets.cpu().numpy(), o)
    assert np.array_equal(r.entry.cpu().numpy(), e)
    assert np.array_equal(r.slot.cpu().numpy(), s)


def _route_fast(ids, K):
    """route_ref for long tables: a stable sort of the keys."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < K), flat, K)
    order = np.argsort(key, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=K + 1)[:K])]).astype(np.int64)
    used = offsets[-1]
    entry = np.full(flat.size, -1, dtype=np.int32)
    entry[:used] = order[:used]
    slot = np.full(flat.size, -1, dtype=np.int32)
    slot[order[:used]] = np.arange(used)
    return offsets, entry, slot.reshape(ids.shape)


def test_route_references_agree():
    rng = np.random.default_rng(1)
    ids = _ids(rng, 500, 3, 40, 0.2)
    for a, b in zip(route_ref(ids, 40), _route_fast(ids, 40)):
        assert np.array_equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("N,m,K", [(3_000_001, 4, 300), (1_500_000, 8, 20_000), (25_000_003, 1, 65_536)])
def test_route_long_tables(cuda, N, m, K):
    """Segments at the length that the 16-bit counts allow, one key in half of
    the entries."""
    import torch
    from soft_clustering_gb300.experts import Router
    rng = np.random.default_rng(K)
    ids = rng.integers(-1, K + 1, (N, m)).astype(np.int32)
    ids[rng.random(N) < 0.5] = K // 2
    r = Router(N, m, K)
    r.route(torch.from_numpy(ids).cuda())
    o, e, s = _route_fast(ids, K)
    assert np.array_equal(r.offsets.cpu().numpy(), o)
    assert np.array_equal(r.entry.cpu().numpy(), e)
    assert np.array_equal(r.slot.cpu().numpy(), s)


@pytest.mark.gpu
def test_route_one_component_takes_all(cuda):
    import torch
    from soft_clustering_gb300.experts import Router
    ids = np.full((70001, 1), 3, dtype=np.int32)
    r = Router(70001, 1, 9)
    r.route(torch.from_numpy(ids).cuda())
    assert r.offsets.cpu().tolist() == [0] * 4 + [70001] * 6
    assert np.array_equal(r.slot.cpu().numpy().reshape(-1), np.arange(70001))


ROWS = [(1, 1, 1, 4), (1, 4, 128, 16), (7, 2, 3, 5), (33, 3, 333, 8), (64, 8, 130, 20), (129, 2, 20, 7),
        (1000, 4, 128, 64), (50, 2, 2048, 8), (300, 4, 1028, 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,m,D,K", ROWS)
def test_spread_and_collect(cuda, dtype, N, m, D, K):
    import torch
    from soft_clustering_gb300.experts import Router
    rng = np.random.default_rng(D + N)
    ids = _ids(rng, N, m, K, 0.2)
    _, entry, slot = route_ref(ids, K)
    r = Router(N, m, K)
    r.route(torch.from_numpy(ids).cuda())
    X, Z = _rand(rng, (N, D), dtype), _rand(rng, (N * m, D), dtype)
    used = int((entry >= 0).sum())
    Z[used:] = float("nan")  # rows of nobody
    gamma = torch.from_numpy(rng.random((N, m)).astype(np.float32)).cuda()
    gamma[torch.from_numpy(slot < 0).cuda()] = float("nan")  # weights of entries left out
    x, z, w = _f64(X), _f64(Z), _f64(gamma)
    rows = entry[:used].astype(np.int64)
    uT, sub = UT[dtype], SUB[dtype]
    # dispatch: equal, and zeros behind
    Y = r.spread(X)
    assert np.array_equal(_f64(Y)[:used], x[rows // m]) and not _f64(Y)[used:].any()
    # with weights and the gradient of gamma
    Y, dg = r.spread(X, gamma, Z)
    ref = np.zeros((N * m, D))
    ref[:used] = x[rows // m] * w.reshape(-1)[rows][:, None]
    _near(Y, ref, (U + uT) * np.abs(ref) + sub, "spread")
    rg, bg = np.zeros(N * m), np.zeros(N * m)
    prod = x[rows // m] * z[:used]
    rg[rows], bg[rows] = prod.sum(1), (D + 1) * U * np.abs(prod).sum(1)
    _near(dg, rg.reshape(N, m), bg.reshape(N, m), "dgamma")
    # combine and the dispatch's gradient
    for wt in (gamma, None):
        out, mag = np.zeros((N, D)), np.zeros((N, D))
        term = z[:used] * (w.reshape(-1)[rows][:, None] if wt is not None else 1.0)
        np.add.at(out, rows // m, term)
        np.add.at(mag, rows // m, np.abs(term))
        _near(r.collect(Z, wt), out, (m + 1) * U * mag + (uT + U) * np.abs(out) * 1.01 + uT * (m + 1) * U * mag + sub,
              "collect")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_rows_at_odd_addresses(cuda, dtype, shift):
    """Every array starts `shift` elements into its storage."""
    import torch
    N, m, D, K = 37, 2, 64, 5
    rng = np.random.default_rng(shift)
    ids = _ids(rng, N, m, K, 0.1)
    o, entry, slot = route_ref(ids, K)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731

    def off(t):
        s = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
        s[shift:] = t.reshape(-1)
        return s[shift:].reshape(t.shape)

    X, Z = off(_rand(rng, (N, D), dtype, True)), off(_rand(rng, (N * m, D), dtype, True))
    Y, out = off(torch.zeros(N * m, D, dtype=_dt(dtype))), off(torch.zeros(N, D, dtype=_dt(dtype)))
    dg = torch.zeros(N, m, device="cuda")
    gam = torch.full((N, m), 2.0, device="cuda")
    so, of = dev(slot), dev(o)
    G.gmm_spread(X, CODE[dtype], N, D, m, K, N * m, so, of, gam, Z, Y, dg)
    G.gmm_collect(Z, CODE[dtype], N, D, m, N * m, so, gam, out)
    used = int(o[-1])
    rows = entry[:used].astype(np.int64)
    assert np.array_equal(_f64(Y)[:used], 2 * _f64(X)[rows // m])
    ref = np.zeros((N, D))
    np.add.at(ref, rows // m, 2 * _f64(Z)[:used])
    assert np.array_equal(_f64(out), ref)


def _offsets(rng, K, R, tail):
    """Uneven rows per component, some with none, `tail` rows of nobody."""
    p = rng.dirichlet(np.full(K, 0.7))
    p[rng.random(K) < 0.2] = 0
    p = p / p.sum() if p.sum() > 0 else np.full(K, 1.0 / K)
    n = rng.multinomial(R - tail, p)
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


PRODUCTS = [(30000, 5, 3, 64, 128), (40000, 0, 5, 256, 40), (9001, 0, 1, 264, 264), (9001, 0, 3, 264, 264), (100, 0, 3, 8, 16), (100, 3, 2, 16, 8), (0, 0, 3, 16, 24), (1, 0, 1, 1, 1), (1, 0, 4, 128, 64), (5, 1, 4, 7, 9), (64, 0, 3, 64, 64),
            (16, 0, 64, 256, 136), (130, 3, 5, 33, 70), (777, 20, 6, 72, 200), (300, 0, 2, 128, 128),
            (1000, 17, 40, 128, 96), (20, 3, 5, 64, 40), (32, 0, 2, 264, 72), (33, 2, 2, 264, 72), (700, 9, 5, 256, 512),
            (90, 0, 9, 1000, 256), (5000, 5, 4000, 64, 40), (5000, 5, 900, 64, 40), (2600, 3, 2, 512, 240), (1500, 40, 60, 240, 256), (7, 7, 3, 16, 8),
            (2500, 0, 3, 320, 264), (513, 1, 1, 1024, 520), (40, 0, 3, 520, 1032)]


def _product_case(rng, R, tail, K, d_in, d_out, dtype, whole):
    import torch
    o = _offsets(rng, K, R, tail)
    used = int(o[-1])
    A, dY = _rand(rng, (R, d_in), dtype, whole), _rand(rng, (R, d_out), dtype, whole)
    A[used:] = float("nan")
    dY[used:] = float("inf")
    W = _rand(rng, (K, d_out, d_in), dtype, whole)
    from soft_clustering_gb300.experts import ExpertProduct
    e = ExpertProduct(K, d_in, d_out, _dt(dtype), R)
    od = torch.from_numpy(o).cuda()
    return e, o, od, used, A, dY, W


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,tail,K,d_in,d_out", PRODUCTS)
def test_product_of_whole_numbers_is_exact(cuda, dtype, R, tail, K, d_in, d_out):
    import torch
    rng = np.random.default_rng(R + K + d_in)
    e, o, od, used, A, dY, W = _product_case(rng, R, tail, K, d_in, d_out, dtype, True)
    a, dy, w = _f64(A), _f64(dY), _f64(W)
    a[used:], dy[used:] = 0, 0
    # rounded once to the type, as numpy -> torch rounds (to nearest, ties to even)
    rnd = lambda x: torch.from_numpy(x).to(torch.float32).to(_dt(dtype)).double().numpy()  # noqa: E731
    assert np.array_equal(_f64(e.forward(A, od, W)), rnd(product_ref(a, w, o)))
    assert np.array_equal(_f64(e.backward_rows(dY, od, W)), rnd(product_ref(dy, w.transpose(0, 2, 1), o)))
    dw = dw_ref(dy, a, o, K)
    assert np.array_equal(_f64(e.backward_weights(dY, A, od)), rnd(dw))
    assert np.array_equal(_f64(e.backward_weights(dY, A, od, out_dtype=torch.float32)), dw)
    assert e.device_status() == G.GMM_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("R,tail,K,d_in,d_out", [(16, 0, 64, 256, 136), (777, 20, 6, 72, 200),
                                                 (2500, 0, 3, 320, 264), (40, 0, 3, 33, 65), (20000, 0, 3, 64, 72), (20000, 0, 5, 64, 72)])
def test_product_of_real_numbers(cuda, dtype, R, tail, K, d_in, d_out):
    import torch
    rng = np.random.default_rng(R)
    e, o, od, used, A, dY, W = _product_case(rng, R, tail, K, d_in, d_out, dtype, False)
    a, dy, w = _f64(A), _f64(dY), _f64(W)
    a[used:], dy[used:] = 0, 0
    uT, sub = UT[dtype], SUB[dtype]

    def check(got, ref, mag, L, u, s, what):
        acc = 2 * L * U * mag
        _near(got, ref, acc + (u + U) * (np.abs(ref) + acc) + s, what)

    wt = w.transpose(0, 2, 1)
    check(e.forward(A, od, W), product_ref(a, w, o), product_ref(abs(a), abs(w), o), d_in, uT, sub, "forward")
    check(e.backward_rows(dY, od, W), product_ref(dy, wt, o), product_ref(abs(dy), abs(wt), o), d_out, uT, sub, "dx")
    L = int(np.diff(o).max()) if K else 0
    ref, mag = dw_ref(dy, a, o, K), dw_ref(abs(dy), abs(a), o, K)
    check(e.backward_weights(dY, A, od), ref, mag, L, uT, sub, "dw")
    check(e.backward_weights(dY, A, od, out_dtype=torch.float32), ref, mag, L, 0.0, 0.0, "dw fp32")


@pytest.mark.gpu
@pytest.mark.parametrize("d_in,d_out", [(128, 128), (72, 200), (264, 64)])
def test_one_component_does_not_reach_another(cuda, d_in, d_out):
    """Infinities and NaN in component 1's rows and weights stay there."""
    import torch
    from soft_clustering_gb300.experts import ExpertProduct
    rng = np.random.default_rng(d_in)
    n = [70, 45, 133]
    o = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    A, dY = _rand(rng, (sum(n), d_in), "bf16", True), _rand(rng, (sum(n), d_out), "bf16", True)
    W = _rand(rng, (3, d_out, d_in), "bf16", True)
    W2, A2, dY2 = W.clone(), A.clone(), dY.clone()
    W2[1] = float("nan")
    A2[70:115] = float("inf")
    dY2[70:115] = float("nan")
    e = ExpertProduct(3, d_in, d_out, torch.bfloat16, sum(n))
    od = torch.from_numpy(o).cuda()
    keep = np.r_[0:70, 115:248]
    for clean, dirty, sel in ((e.forward(A, od, W), e.forward(A2, od, W2), keep),
                              (e.backward_rows(dY, od, W), e.backward_rows(dY2, od, W2), keep),
                              (e.backward_weights(dY, A, od), e.backward_weights(dY2, A2, od), [0, 2])):
        assert np.array_equal(_f64(clean)[sel], _f64(dirty)[sel])


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 8])
def test_product_at_odd_addresses(cuda, shift):
    import torch
    rng = np.random.default_rng(5)
    R, K, d_in, d_out = 150, 3, 64, 128
    e, o, od, used, A, dY, W = _product_case(rng, R, 0, K, d_in, d_out, "f16", True)

    def off(t):
        s = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
        s[shift:] = t.reshape(-1)
        return s[shift:].reshape(t.shape)

    a, dy, w = _f64(A), _f64(dY), _f64(W)
    zero = lambda *s: off(torch.zeros(*s, dtype=torch.float16))  # noqa: E731
    assert np.array_equal(_f64(e.forward(off(A), od, off(W), out=zero(R, d_out))), product_ref(a, w, o))
    assert np.array_equal(_f64(e.backward_rows(off(dY), od, off(W), out=zero(R, d_in))),
                          product_ref(dy, w.transpose(0, 2, 1), o))
    assert np.array_equal(_f64(e.backward_weights(off(dY), off(A), od, out=zero(K, d_out, d_in))), dw_ref(dy, a, o, K))


@pytest.mark.gpu
def test_elements_past_32_bits(cuda):
    """More than 2^31 elements of rows, and of weights."""
    import torch
    from soft_clustering_gb300.experts import ExpertProduct, Router
    N, m, K, D = 1_100_000, 1, 600, 2048
    ids = (torch.arange(N, device="cuda", dtype=torch.int32) % K).reshape(N, 1)
    X = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = (torch.arange(N, device="cuda") % 251).to(torch.bfloat16)
    r = Router(N, m, K)
    r.route(ids)
    Y = r.spread(X)
    assert torch.equal(Y[r.slot[:, 0].long(), 0], X[:, 0])
    W = torch.zeros(K, D, D, dtype=torch.bfloat16, device="cuda")
    W[:, 0, 0] = (torch.arange(K, device="cuda") % 97).to(torch.bfloat16)
    W[:, D - 1, 0] = 1.0
    o = torch.arange(K + 1, device="cuda") * 3
    A = Y[N - 3 * K:].contiguous()
    e = ExpertProduct(K, D, D, torch.bfloat16, 3 * K)
    out = e.forward(A, o, W)
    a = A[:, 0].float()
    ref = (a * W[:, 0, 0].float().repeat_interleave(3)).to(torch.bfloat16)
    assert torch.equal(out[:, 0], ref) and torch.equal(out[:, D - 1], A[:, 0])
    assert not out[:, 1:D - 1].any()
    dW = e.backward_weights(A, A, o)
    assert torch.equal(dW[:, 0, 0], (a * a).reshape(K, 3).sum(1).to(torch.bfloat16))
    out = r.collect(Y)
    assert torch.equal(out[:, 0], X[:, 0])


@pytest.mark.gpu
def test_another_stream_and_repeatability(cuda):
    import torch
    from soft_clustering_gb300.experts import LocalExperts
    rng = np.random.default_rng(2)
    N, m, K, d = 900, 2, 12, 128
    ids = torch.from_numpy(_ids(rng, N, m, K, 0.1)).cuda()
    gam = torch.from_numpy(rng.random((N, m)).astype(np.float32)).cuda()
    X, W, g = _rand(rng, (N, d), "bf16"), _rand(rng, (K, d, d), "bf16"), _rand(rng, (N, d), "bf16")
    layer = LocalExperts(N, m, K, d, d, torch.bfloat16)
    torch.cuda.synchronize()
    first = [layer.forward(X, ids, gam, W), *layer.backward(g, W)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again = [layer.forward(X, ids, gam, W, stream=s), *layer.backward(g, W, stream=s)]
    s.synchronize()
    with torch.cuda.stream(s):
        third = [layer.forward(X, ids, gam, W), *layer.backward(g, W)]
    s.synchronize()
    for a, b, c in zip(first, again, third):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
def test_gradients_against_differences(cuda):
    """L = <c, layer(X, gamma, W)> is linear in each of X, gamma and W, so a
    central difference of any step has rounding error alone: each L is a sum of
    N m d_in d_out products in fp32, off by at most (number of roundings of a
    path) u sum |terms|."""
    import torch
    from soft_clustering_gb300.experts import LocalExperts
    rng = np.random.default_rng(4)
    N, m, K, di, do = 9, 3, 4, 10, 6
    ids = torch.from_numpy(_ids(rng, N, m, K, 0.1)).cuda()
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    X, W, c = t(N, di), t(K, do, di), t(N, do)
    gam = torch.from_numpy(rng.random((N, m)).astype(np.float32)).cuda()
    layer = LocalExperts(N, m, K, di, do, torch.float32)

    def loss(X, gam, W):
        return float((layer.forward(X, ids, gam, W).double() * c.double()).sum())

    size = float(layer.forward(X.abs(), ids, gam, W.abs()).double().mul(c.abs().double()).sum())
    layer.forward(X, ids, gam, W)
    grads = layer.backward(c, W)
    h = 0.5
    bound = 2 * (2 * (di + do + m + 4)) * U * size / h
    for which, (v, g) in enumerate(zip((X, gam, W), grads)):
        for i in rng.choice(v.numel(), 12, replace=False):
            up, dn = v.clone(), v.clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            args = [X, gam, W]
            vals = []
            for x in (up, dn):
                args[which] = x
                vals.append(loss(*args))
            # the perturbed value itself is rounded: use the steps as taken
            step = float(up.view(-1)[i].double() - dn.view(-1)[i].double())
            fd = (vals[0] - vals[1]) / step
            assert abs(fd - float(g.reshape(-1)[i])) <= bound * 2, (which, i, fd, float(g.reshape(-1)[i]), bound)


@pytest.mark.gpu
def test_python_refusals(cuda):
    import torch
    from soft_clustering_gb300.experts import ExpertProduct, LocalExperts, Router
    with pytest.raises(ValueError):
        Router(10, 9, 4)
    with pytest.raises(ValueError):
        ExpertProduct(4, 0, 8, torch.float16, 10)
    with pytest.raises(ValueError):
        ExpertProduct(4, 8, 8, torch.float64, 10)
    r = Router(6, 2, 4)
    with pytest.raises(ValueError):
        r.route(torch.zeros(6, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        r.route(torch.zeros(6, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        r.route(torch.zeros(2, 6, dtype=torch.int32, device="cuda").t())
    with pytest.raises(ValueError):
        r.spread(torch.zeros(5, 8, device="cuda"))
    with pytest.raises(ValueError):
        r.spread(torch.zeros(6, 8, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        r.spread(torch.zeros(6, 16, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        r.collect(torch.zeros(12, 8, device="cuda"), gamma=torch.zeros(6, 2, device="cuda").half())
    e = ExpertProduct(4, 8, 16, torch.float16, 12)
    o = torch.zeros(5, dtype=torch.int64, device="cuda")
    W = torch.zeros(4, 16, 8, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        e.forward(torch.zeros(13, 8, dtype=torch.float16, device="cuda"), o, W)
    with pytest.raises(ValueError):
        e.forward(torch.zeros(12, 8, dtype=torch.float16, device="cuda"), o, W.transpose(1, 2))
    with pytest.raises(ValueError):
        e.backward_weights(torch.zeros(12, 16, dtype=torch.float16, device="cuda"),
                           torch.zeros(11, 8, dtype=torch.float16, device="cuda"), o)
    with pytest.raises(RuntimeError):
        LocalExperts(2, 1, 2, 8, 8, torch.float16).backward(torch.zeros(2, 8, device="cuda").half(), W)


@pytest.mark.gpu
@pytest.mark.parametrize("state_bits", [8, 32])
def test_mixture_of_local_experts_learns(cuda, state_bits):
    """The example end to end: EM, gate, experts, gradients, AdamW.  Answers that
    are linear within each component are recovered to a small part of their
    variance (bf16 products: relative error near 2^-8)."""
    import importlib.util
    import os
    p = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "local_experts.py")
    spec = importlib.util.spec_from_file_location("local_experts", p)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(N=6000, K=8, steps=120, state_bits=state_bits, log=None)
    assert all(np.isfinite(losses)) and losses[-1] < 0.05 * losses[0], (losses[0], losses[-1])


@pytest.mark.gpu
def test_captured_in_a_graph(cuda):
    """Forward, backward and the weights' step replayed from a CUDA graph."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    from soft_clustering_gb300.experts import LocalExperts
    rng = np.random.default_rng(8)
    N, m, K, d = 700, 2, 10, 256
    ids = torch.from_numpy(_ids(rng, N, m, K, 0.1)).cuda()
    gam = torch.from_numpy(rng.random((N, m)).astype(np.float32)).cuda()
    X, g = _rand(rng, (N, d), "bf16"), _rand(rng, (N, d), "bf16")
    W0 = _rand(rng, (K, d, d), "bf16")

    def build():
        W = W0.clone()
        return W, LocalExperts(N, m, K, d, d, torch.bfloat16), AdamW([W], state_bits=8)

    def once(W, layer, opt):
        out = layer.forward(X, ids, gam, W)
        dX, dg, dW = layer.backward(g, W)
        opt.step([dW])
        return out, dX, dg, dW

    a = build()
    eager = [t.clone() for t in once(*a)] + [a[0].clone()]
    b = build()
    once(*b)
    W, layer, opt = b
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.steps = 0  # the captured step is step 1
        outs = once(*b)
    W.copy_(W0)
    for k, ts in opt.state.items():
        for t in ts:
            t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(eager, [*outs, W]):
        assert torch.equal(x, y)
