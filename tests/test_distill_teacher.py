"""Distillation where a teacher's values, or the temperature, are at the ends of
what is allowed.

Tolerances are test_gate.py's, but for the teacher's share q: of logits a value
less the row's largest has one rounding, times log2 e / T three more, and exp2 is
within 2^-21, so that q goes by an entry's distance from the largest alone:
relq = 4 u spread + 2^-20 + 300 u.
"""
import numpy as np
import pytest

import soft_clustering_gb300 as G
from test_gate import SUB, U, UT, _E, _S, _f64, _logits, _misaligned, _near, distill_ref, softmax_ref

# lanes of a warp with an entry each and with eight, all of it, a block, streamed, shared by blocks
FORMS = [(12, 8, 4), (300, 40, 20), (40, 64, 40), (33, 101, 9), (50, 256, 4), (70, 500, 33), (20, 1024, 32),
         (20, 1024, 64), (30, 1025, 5), (20, 4096, 40), (100, 9001, 7), (90, 50257, 32), (10, 50257, 64)]


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def _check(L, ids, vals, kind, T, dtype, relq_of, shifted=False, scale=0.25):
    """rows, loss and gradient of the kernels against the restatement."""
    import torch
    from soft_clustering_gb300.gate import Distiller
    x = _f64(L)
    N, K = x.shape
    m = ids.shape[1]
    w = np.ones(N)
    ref, loss, rd, p, q, u, on = distill_ref(x, ids, vals.astype(float), kind, T, w, scale)
    if shifted:
        L = _misaligned(L)
    d = Distiller(N, K, m, L.dtype, teacher=kind, temperature=T, scale=scale)
    total, got = d.step(L, torch.from_numpy(ids).cuda(), torch.from_numpy(vals).cuda(),
                        out=_misaligned(torch.full_like(L, 5.0)) if shifted else None)
    _, _, a = softmax_ref(x / T)
    S = _S(p, a)
    with np.errstate(invalid="ignore"):
        top = np.where(np.isfinite(u), u, -np.inf).max(1, keepdims=True)
        spread = np.where(q > 0, np.abs(u - top), 0.0)
    relq = relq_of(u, spread)
    at = np.where((ids >= 0) & (ids < K), ids, 0)
    la = np.where(q > 0, np.abs(np.take_along_axis(a, at, 1)), 0.0)
    size = 1 + (q * (spread + la)).sum(1) + np.log(np.exp(a).sum(1))
    br = np.where(on, T * T * ((relq * q).sum(1) + S[:, 0] + 64 * U) * size, 0.0) + 2.0 ** -126
    _near(d.rows, ref, br, "rows")
    _near(total, np.array([loss]), scale * br.sum() + 2 * U * abs(loss), "loss")
    big = scale * T * p * (_E(a) + S + 12 * U)
    peak = scale * T * q * (relq + 8 * U)
    for t in range(m):
        r = np.nonzero(q[:, t] > 0)[0]
        big[r, ids[r, t]] += peak[r, t]
    _near(got, rd, big + (UT[dtype] + 4 * U) * np.abs(rd) + SUB[dtype], "dlogits")


def _apart(rng, N, K, m):
    """m different entries a row."""
    return np.stack([rng.permutation(K)[:m] for _ in range(N)]).astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,m", FORMS)
def test_teacher_far_from_zero(cuda, N, K, m, dtype):
    """A number that all of a row's values have in common is of no consequence, and
    the type's lowest is a value as any other: rows of it alone have even shares."""
    rng = np.random.default_rng(K + m)
    L = _logits(rng, N, K, dtype, plain=True)
    ids = _apart(rng, N, K, m)
    # multiples of 1/16 up to 6: exact beside the offsets
    vals = rng.integers(0, 96, (N, m)) / 16.0
    low = float(np.finfo(np.float32).min)
    offsets = [0.0, 1e3, -1e3, 1e4, -1e4, 2.0 ** 19, -(2.0 ** 19)]
    vals = (vals + np.array([offsets[n % len(offsets)] for n in range(N)])[:, None]).astype(np.float32)
    vals[1] = low
    vals[2, m // 2:] = low
    vals[3] = -low
    vals[4, : m - 1] = -np.inf
    vals[5] = low
    vals[5, 0] = -low
    ids[6] = -1
    if m > 2:
        ids[7, 1], ids[7, 2] = K, -1
        vals[7, 1:3] = np.nan  # of no entry
    relq = lambda u, spread: 4 * U * spread + 2.0 ** -20 + 300 * U  # noqa: E731
    for T, shifted in ((1.0, False), (0.5, True), (3.0, False)):
        _check(L, ids, vals, "logits", T, dtype, relq, shifted)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,m", FORMS)
def test_small_gammas(cuda, N, K, m):
    """Shares below 2^-126 are shares: large where the temperature is, and where all
    of a row are as small.

    The log of a share s is within 2^-21 |log s|: so its power within 2^-20 of the
    exponents, at most 104 / T."""
    rng = np.random.default_rng(K + m)
    L = _logits(rng, N, K, "f32", plain=True)
    ids = _apart(rng, N, K, m)
    with np.errstate(under="ignore"):
        vals = (10.0 ** rng.uniform(-44, 0, (N, m))).astype(np.float32)
    vals[1] = np.float32(1e-40) * (1 + np.arange(m) % 3)
    vals[2] = np.float32(1.4e-45)
    vals[3] = 0.0
    vals[4, 0] = 0.0
    for T, shifted in ((1.0, False), (50.0, True), (1000.0, False)):
        _check(L, ids, vals, "gamma", T, "f32",
               lambda u, spread: 2.0 ** -20 * np.where(np.isfinite(u), np.abs(u), 0.0).max(1, keepdims=True)
               + 4 * U * spread + 2.0 ** -20 + 300 * U, shifted)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,m", FORMS)
def test_small_temperatures(cuda, N, K, m):
    """T^2 is below 2^-126 where T times the logits is not."""
    rng = np.random.default_rng(K + m)
    L = _logits(rng, N, K, "f32", plain=True)
    ids = _apart(rng, N, K, m)
    vals = (rng.standard_normal((N, m))).astype(np.float32)
    for T in (1e-12, 2.0 ** -80, 1e-30):
        _check(L, ids, vals, "logits", T, "f32", lambda u, spread: 4 * U * spread + 2.0 ** -20 + 300 * U, scale=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,m", FORMS)
def test_a_masked_student_at_the_teachers_entry(cuda, N, K, m):
    """The lowest number is far away, not infinitely far, whatever the temperature."""
    rng = np.random.default_rng(K + m)
    L = _logits(rng, N, K, "f32", plain=True)
    ids = _apart(rng, N, K, m)
    low = float(np.finfo(np.float32).min)
    import torch
    L[torch.arange(N, device="cuda"), torch.from_numpy(ids[:, 0].astype(np.int64)).cuda()] = low
    vals = np.full((N, m), 1.0, dtype=np.float32)
    for T in (1.0, 0.5, 0.01):
        _check(L, ids, vals, "gamma", T, "f32", lambda u, spread: 2.0 ** -20 + 300 * U, scale=2.0 ** -10)


def test_temperatures_whose_inverse_is_no_number_are_refused():
    from soft_clustering_gb300 import build
    build.build()
    P = 4096
    for T in (1e-45, 1e-39, 3e-39, 4e38, 1e300):
        assert G.lib().gmm_distill(P, 1, 10, 64, 2, 0, 0, T, 1.0, P, P, P, P, P, P, P, 1 << 40,
                                   None) == G.GMM_ERR_INVALID_ARG, T
