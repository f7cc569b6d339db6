"""AdamW as programs use it: storage that moves, state that is loaded, other
streams, graphs, values that are not finite, long schedules.

Every comparison is with the same step taken another way, equal to the bit,
unless a test derives its bound.
"""
import numpy as np
import pytest

import soft_clustering_gb300 as G


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
