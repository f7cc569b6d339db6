"""Local experts as programs use them: batches that overlap, buffers that are
written again, other streams, neighbours that are not finite.

References and tolerances are those of test_experts.py: products of small whole
numbers are exact, and what is compared with itself has to be equal.
"""
import numpy as np
import pytest

import soft_clustering_gb300 as G
from test_experts import _f64, _ids, _rand, dw_ref


@pytest.fixture(scope="module")
def lib():
    from soft_clustering_gb300 import build
    build.build()
    return G.lib()


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from soft_clustering_gb300 import build
    build.build()
    return torch.device("cuda", 0)


@pytest.mark.gpu
@pytest.mark.parametrize("d_in,d_out", [(64, 256), (264, 512), (512, 240)])
def test_ragged_ends_in_pairs_of_blocks(cuda, d_in, d_out):
    """dW where two blocks share a tile and every component ends inside a stage:
    the rows of the next component, infinities and NaN, reach no sum, time after
    time."""
    import torch
    from soft_clustering_gb300.experts import ExpertProduct
    rng = np.random.default_rng(d_out)
    n = [1, 15, 17, 63, 65, 127, 40, 200, 3, 90] * 8
    o = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    K, R = len(n), sum(n)
    A, dY = _rand(rng, (R, d_in), "bf16", True), _rand(rng, (R, d_out), "bf16", True)
    odd = np.repeat(np.arange(K) % 2 == 1, n)
    ref = dw_ref(_f64(dY), _f64(A), o, K)[::2]
    A[torch.from_numpy(odd).cuda()] = float("inf")
    dY[torch.from_numpy(odd).cuda()] = float("nan")
    e = ExpertProduct(K, d_in, d_out, torch.bfloat16, R)
    od = torch.from_numpy(o).cuda()
    for _ in range(20):
        dW = e.backward_weights(dY, A, od, out_dtype=torch.float32)
        assert np.array_equal(_f64(dW[::2]), ref)
        assert torch.isnan(dW[1::2]).all()
    assert e.device_status() == G.GMM_OK


def _layer(seed=0, N=300, m=2, K=6, d=64, drop=0.1):
    import torch
    from soft_clustering_gb300.experts import LocalExperts
    rng = np.random.default_rng(seed)
    ids = torch.from_numpy(_ids(rng, N, m, K, drop)).cuda()
    gam = torch.from_numpy(rng.random((N, m)).astype(np.float32)).cuda()
    X, W, c = _rand(rng, (N, d), "bf16"), _rand(rng, (K, d, d), "bf16"), _rand(rng, (N, d), "bf16")
    return ids, gam, X, W, c, LocalExperts(N, m, K, d, d, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("side", [False, True])
def test_gate_buffers_written_between_forward_and_backward(cuda, side):
    """The next batch's ids and gamma in the buffers that forward was given."""
    import torch
    ids, gam, X, W, c, layer = _layer()
    s = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    layer.forward(X, ids, gam, W)
    want = layer.backward(c, W)
    torch.cuda.synchronize()
    layer.forward(X, ids, gam, W, stream=s)
    torch.cuda.synchronize()
    gam.fill_(float("nan"))
    ids.fill_(3)
    torch.cuda.synchronize()
    got = layer.backward(c, W, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_backward_of_rows_that_lost_their_places(cuda):
    """Other ids in the layer's router, or a forward that failed half way: no
    backward pass of the rows before."""
    import torch
    ids, gam, X, W, c, layer = _layer()
    other = ids.flip(0).contiguous()
    want = layer.forward(X, ids, gam, W)
    layer.router.route(other)
    with pytest.raises(RuntimeError):
        layer.backward(c, W)
    assert torch.equal(layer.forward(X, ids, gam, W), want)
    layer.backward(c, W)
    for bad in ((X, other, gam, W[:, :, :32].contiguous()), (X.float(), other, gam, W)):
        layer.forward(X, ids, gam, W)
        with pytest.raises(ValueError):
            layer.forward(*bad)
        with pytest.raises(RuntimeError):
            layer.backward(c, W)
    layer.forward(X, ids, gam, W)
    with pytest.raises(ValueError):  # refused before anything changed
        layer.forward(X, other, gam[:, :1], W)
    layer.backward(c, W)


@pytest.mark.gpu
def test_kept_rows_outlive_a_backward_on_another_stream(cuda):
    """Memory of the kept rows is not handed out again while a backward pass on
    another stream may still read it."""
    import torch
    ids, gam, X, W, c, layer = _layer()
    layer.forward(X, ids, gam, W)
    want = [t.clone() for t in layer.backward(c, W)]
    layer.forward(X, ids, gam, W)
    shape, side = layer._kept[0].shape, torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second
        got = layer.backward(c, W)
    layer._kept = None  # as the next forward does first
    taken = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert len(taken) == 4
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,N,K,d", [("bf16", 300, 6, 64), ("bf16", 4, 20, 64), ("bf16", 900, 1500, 256),
                                         ("bf16", 20000, 3, 64), ("f32", 60, 4, 24), ("f16", 0, 4, 64)])
def test_a_failure_outlives_the_products_after_it(cuda, dtype, N, K, d):
    """A status raised in one product is there after the others, in every form
    of the product, until it is cleared."""
    import torch
    from soft_clustering_gb300.experts import LocalExperts
    rng = np.random.default_rng(N)
    ids = torch.from_numpy(rng.integers(0, K, (N, 1)).astype(np.int32)).cuda()
    X, W, c = _rand(rng, (N, d), dtype), _rand(rng, (K, d, d), dtype), _rand(rng, (N, d), dtype)
    layer = LocalExperts(N, 1, K, d, d, X.dtype)
    gam = torch.ones(N, 1, device="cuda")

    def step():
        layer.forward(X, ids, gam, W)
        layer.backward(c, W)

    step()
    assert layer.device_status() == G.GMM_OK
    layer.product.ws[:4].view(torch.int32).fill_(G.GMM_ERR_TIMEOUT)
    step()
    assert layer.device_status() == G.GMM_ERR_TIMEOUT
    layer.product.clear_status()
    step()
    assert layer.device_status() == G.GMM_OK


def test_only_the_current_cuda_device(monkeypatch):
    """The launch goes to the current device: other tensors are refused before
    it, on the host or on another GPU."""
    import torch
    from soft_clustering_gb300 import adamw, experts
    for make in (lambda: experts.Router(4, 2, 3, device="cpu"),
                 lambda: experts.ExpertProduct(3, 8, 8, torch.float16, 4, device="cpu"),
                 lambda: experts.LocalExperts(4, 2, 3, 8, 8, torch.float16, device="cpu")):
        with pytest.raises(ValueError, match="CUDA device"):
            make()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    experts._here(torch.device("cuda", 0))
    with pytest.raises(ValueError, match="current device"):
        experts._here(torch.device("cuda", 1))

    # every call looks: objects of another device, as they would be there
    other = torch.device("cuda", 1)
    monkeypatch.setattr(experts, "_need", lambda t, *a: t)
    x = torch.zeros(4, 8, dtype=torch.float16)
    r, e, o = (object.__new__(c) for c in (experts.Router, experts.ExpertProduct, adamw.AdamW))
    r.N, r.m, r.rows, r.K, r.device = 4, 1, 4, 3, other
    e.max_rows, e.dtype, e.device, e.d_in, e.d_out = 4, torch.float16, other, 8, 8
    e._offsets_shape = e._w_shape = None
    o.params, o._device = [x], other
    for call in (lambda: r.route(x), lambda: r.spread(x), lambda: r.collect(x), lambda: e.forward(x, x, x),
                 lambda: e.backward_rows(x, x, x), lambda: e.backward_weights(x, x, x), lambda: o.step([x]),
                 lambda: o.moments()):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_addresses_that_are_not_aligned(lib):
    """Refused before anything is queued, for every array of every call."""
    bad, P, big = G.GMM_ERR_INVALID_ARG, 4096, 1 << 40

    def each(f, args, where):
        for i, by in where.items():
            a = list(args)
            a[i] += by
            assert f(*a) == bad, (f.__name__, i)

    each(lib.gmm_route, (P, 10, 2, 4, P, P, P, P, big, None), {0: 2, 4: 4, 5: 1, 6: 2, 7: 2})
    each(lib.gmm_spread, (P, 1, 5, 8, 2, 3, 10, P, P, P, P, P, P, None), {0: 1, 7: 2, 8: 4, 9: 2, 10: 1, 11: 1, 12: 2})
    each(lib.gmm_collect, (P, 1, 5, 8, 2, 10, P, P, P, None), {0: 1, 6: 2, 7: 1, 8: 1})
    for f in (lib.gmm_expert_product, lib.gmm_expert_product_dx):
        each(f, (P, 1, 4, 8, 8, 2, P, P, P, P, big, None), {0: 1, 6: 4, 7: 1, 8: 1, 9: 128})
    each(lib.gmm_expert_product_dw, (P, P, 1, 4, 8, 8, 2, P, P, 0, P, big, None), {0: 1, 1: 1, 7: 4, 8: 2, 10: 128})


def test_workspace_holds_what_the_product_uses(lib):
    """Partial sums of dW only where the tensor cores can make them, and never
    less for fewer rows of the same product."""
    R, K = 522711, 22
    part = 4 * 64 * 128 * 100  # a hundred partial sums at least
    assert G.gmm_expert_ws_bytes(R, 64, 128, K, G.GMM_BF16) > part
    for d_in, d_out, x in ((64, 128, G.GMM_F32), (60, 128, G.GMM_BF16), (64, 124, G.GMM_F16)):
        assert G.gmm_expert_ws_bytes(R, d_in, d_out, K, x) < part
    for x in (G.GMM_F32, G.GMM_F16):
        for d_in, d_out, K in ((64, 128, 22), (512, 256, 16), (8, 8, 1), (128, 128, 600), (2048, 2048, 3)):
            sizes = [G.gmm_expert_ws_bytes(r, d_in, d_out, K, x) for r in range(0, 4_000_000, 4093)]
            assert sizes == sorted(sizes) and sizes[0] > 0
