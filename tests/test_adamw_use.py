"""AdamW as programs use it: storage that moves, state that is loaded, other
streams, graphs, values that are not finite, long schedules.

Every comparison is with the same step taken another way, equal to the bit,
unless a test derives its bound.
"""
import ctypes

import numpy as np
import pytest

import soft_clustering_gb300 as G


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


def _make(n=(1000, 300), bits=32, dtype="float32", master=False, seed=0):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    p = [torch.randn(k, device="cuda", generator=g).to(getattr(torch, dtype)) for k in n]
    grads = [[torch.randn(k, device="cuda", generator=g) for k in n] for _ in range(3)]
    return p, grads, AdamW(p, lr=0.1, state_bits=bits, master=master)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
def test_parameters_with_new_storage(cuda, bits, master):
    """The step goes to a parameter's storage of the moment, and nothing is
    written to what it had before."""
    import torch
    want, grads, opt = _make(bits=bits, dtype="bfloat16", master=master)
    for g in grads:
        opt.step(g)
    p, grads, opt = _make(bits=bits, dtype="bfloat16", master=master)
    opt.step(grads[0])
    for q in p:
        q.old = q.data
        q.data = q.data.clone()
    kept = [q.old.clone() for q in p]
    opt.step(grads[1])
    opt.params[1] = p[1].clone()  # another tensor altogether
    opt.step(grads[2])
    assert torch.equal(p[0], want[0]) and torch.equal(opt.params[1], want[1])
    for q, k in zip(p, kept):
        assert torch.equal(q.old, k)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_state_that_is_replaced(cuda, bits):
    """A checkpoint put into a live optimiser's lists, or into the tensors'
    storage, is what the next step and `moments` read."""
    import torch
    want, grads, one = _make(bits=bits, dtype="bfloat16", master=True)
    one.step(grads[0])
    saved = {k: [t.clone() for t in ts] for k, ts in one.state.items()}
    at = [q.clone() for q in want]
    one.step(grads[1])
    m1, v1 = one.moments()
    p, _, two = _make(bits=bits, dtype="bfloat16", master=True, seed=9)
    two.step(grads[2])
    before = {k: list(ts) for k, ts in two.state.items()}
    kept = {k: [t.clone() for t in ts] for k, ts in before.items()}
    for k, ts in saved.items():
        two.state[k][0] = ts[0]
        two.state[k] = [two.state[k][0], ts[1]]
    for q, a in zip(p, at):
        q.copy_(a)
    two.steps = 1
    two.step(grads[1])
    m2, v2 = two.moments()
    for a, b in zip([*want, *m1, *v1], [*p, *m2, *v2]):
        assert torch.equal(a, b)
    for k in before:  # what the lists held before is left alone
        for a, b in zip(before[k], kept[k]):
            assert torch.equal(a, b), k


@pytest.mark.gpu
def test_changes_that_are_refused(cuda):
    import torch
    p, grads, opt = _make()

    def refused(change, back):
        change()
        kept = [t.clone() for t in (*p, *opt.state["v"])]
        with pytest.raises(ValueError):
            opt.step(grads[0])
        with pytest.raises(ValueError):
            opt.moments()
        assert opt.steps == 0
        for a, b in zip(kept, (*p, *opt.state["v"])):
            assert torch.equal(a, b)
        back()

    data, m = p[0].data, opt.state["m"][0]
    put = lambda t: (lambda: setattr(p[0], "data", t))  # noqa: E731
    state = lambda t: (lambda: opt.state["m"].__setitem__(0, t))  # noqa: E731
    for t in (data[:999], data.bfloat16(), data.cpu(), torch.zeros(2000, device="cuda")[::2]):
        refused(put(t), put(data))
    for t in (m[:999], m.half(), m.cpu(), torch.zeros(2000, device="cuda")[::2], None):
        refused(state(t), state(m))
    refused(lambda: opt.params.append(p[0]), opt.params.pop)
    opt.step(grads[0])
    assert opt.steps == 1


@pytest.mark.gpu
def test_autograd_sees_the_step(cuda):
    """A backward pass that saved the parameter before the step refuses."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    w = torch.ones(8, device="cuda", requires_grad=True)
    x = torch.ones(8, device="cuda", requires_grad=True)
    y = (w * x).sum()
    AdamW([w]).step([torch.ones(8, device="cuda")])
    with pytest.raises(RuntimeError):
        y.backward()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), -float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("at,n", [(300, 1024), (0, 256), (511, 700), (699, 700)])
def test_gradients_that_are_not_finite(cuda, bad, dtype, at, n):
    """32 bits: the element alone.  8 bits: its parameter at once, both moments
    of its block, and nothing else."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    block = slice(at // 256 * 256, min(n, at // 256 * 256 + 256))
    for bits in (32, 8):
        p = torch.zeros(n, device="cuda")
        opt = AdamW([p], state_bits=bits)
        opt.step([torch.linspace(-1, 1, n, device="cuda").to(getattr(torch, dtype))])
        g = torch.ones(n, device="cuda", dtype=getattr(torch, dtype))
        g[at] = bad
        opt.step([g])
        hit = torch.zeros(n, dtype=torch.bool, device="cuda")
        hit[at] = True
        assert torch.equal(~torch.isfinite(p), hit)
        if bits == 8:
            hit[block] = True
        for x in opt.moments():
            assert torch.equal(~torch.isfinite(x[0]), hit)
            if bits == 8:
                assert torch.isnan(x[0][block]).all()
        opt.step([torch.ones(n, device="cuda")])
        assert torch.equal(~torch.isfinite(p), hit)
        assert torch.equal(~torch.isfinite(opt.moments()[0][0]), hit)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_moments_on_another_stream(cuda, bits):
    """Outputs that `moments` makes for another stream are not memory that the
    current one still writes."""
    import torch
    n = 1 << 20
    p, _, opt = _make(n=(n,), bits=bits)
    opt.step([torch.ones(n, device="cuda")])
    want = [t[0].clone() for t in opt.moments()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    x = [torch.empty(n, device="cuda") for _ in range(2)]
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    for t in x:
        t.fill_(3.0)
    del x, t
    got = opt.moments(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b[0])


def test_refusals_of_the_counted_step(lib):
    e = (G.gmm_adamw_tensor * 1)(G.gmm_adamw_tensor(param=256, grad=256, m=256, v=256, n=8))
    o = lambda **k: ctypes.byref(G.gmm_adamw_opts(**{**dict(  # noqa: E731
        lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, state_bits=32), **k}))
    call = lambda steps, **k: lib.gmm_adamw_step_counted(e, 1, o(**k), steps, None)  # noqa: E731
    assert call(None) == G.GMM_ERR_INVALID_ARG
    assert call(260) == G.GMM_ERR_INVALID_ARG
    assert lib.gmm_adamw_step_counted(e, 1, None, 256, None) == G.GMM_ERR_INVALID_ARG
    assert lib.gmm_adamw_step_counted(None, 1, o(), 256, None) == G.GMM_ERR_INVALID_ARG
    for bad in (dict(beta1=1.0), dict(beta2=-0.5), dict(lr=float("nan")), dict(state_bits=8)):
        assert call(256, **bad) == G.GMM_ERR_INVALID_ARG, bad


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [("float32", False), ("bfloat16", True), ("float16", False)])
@pytest.mark.parametrize("grad", ["float32", "bfloat16"])
def test_replays_count_their_steps(cuda, bits, dtype, master, grad):
    """A captured step that counts on the device: every replay is the next step,
    equal to the same steps without a graph.  Against the step counted on the
    host the moments are equal; the two corrections are each the rounding of a
    double that may differ in its last place, so one unit of fp32 apart, 2^-23 of
    the update each, and its at most six operations round differently: 2^-20 of
    an update of at most 10 lr (the first steps' moments are of one size), and
    2^-23 of the parameter for its own two roundings, a step."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    dt, lr, steps = getattr(torch, dtype), 0.01, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n = (3000, 17, 600)
    p0 = [torch.randn(k, device="cuda", generator=g).to(dt) for k in n]
    grads = [[torch.randn(k, device="cuda", generator=g).to(getattr(torch, grad)) for k in n] for _ in range(steps)]

    def made(**kw):
        p = [t.clone() for t in p0]
        return p, AdamW(p, lr=lr, state_bits=bits, master=master, **kw)

    p, opt = made(capturable=True)
    q, eager = made(capturable=True)
    r, host = made()
    buf = [t.clone() for t in grads[0]]
    opt.step(buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(buf)
    for x in grads[1:]:
        for b, t in zip(buf, x):
            b.copy_(t)
        graph.replay()
    for x in grads:
        eager.step(x)
        host.step(x)
    assert opt.steps == eager.steps == host.steps == steps
    same = lambda a, b: all(torch.equal(x, y) for k in a.state for x, y in zip(a.state[k], b.state[k])  # noqa: E731
                            if x is not None and k != "master")
    assert same(opt, eager) and same(opt, host)
    for a, b in zip(p, q):
        assert torch.equal(a, b)
    if dtype != "float16":  # held in fp32
        get = lambda o, w: w if dtype == "float32" else o.state["master"]  # noqa: E731
        for a, b in zip(get(opt, p), get(host, r)):
            bound = steps * (2.0 ** -20 * 10 * lr + 2.0 ** -23 * (b.abs() + 10 * lr * steps))
            assert ((a - b).abs() <= bound).all()


@pytest.mark.gpu
def test_steps_of_a_counted_optimiser(cuda):
    """Set, resumed, and counted where a step is skipped."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    p = torch.zeros(8, device="cuda")
    opt = AdamW([p], capturable=True, step=3)
    assert opt.steps == 3
    opt.step([p.clone()], skip=torch.ones(1, dtype=torch.int32, device="cuda"))
    assert opt.steps == 4 and not p.any()
    opt.steps = 10
    opt.step([torch.ones_like(p)])
    assert opt.steps == 11 and p.all()


@pytest.mark.gpu
def test_capture_with_a_fixed_step_warns(cuda):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    p, g = torch.zeros(8, device="cuda"), torch.ones(8, device="cuda")
    opt = AdamW([p])
    opt.step([g])
    with pytest.warns(UserWarning, match="capturable"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            opt.step([g])
