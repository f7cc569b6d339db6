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


# ------------------------------------------------- 8-bit moments, seeded codes

def _philox(c, k):
    """Philox4x32-10 of counters c [..., 4] and a key of two words, in numpy."""
    c = [c[..., i].astype(np.uint64) for i in range(4)]
    k0, k1, low = k[0], k[1], np.uint64(0xffffffff)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return np.stack(c, -1)


def _uniform(n, step, tensor, which):
    """The sixteen bits of each of n elements as (h + 1/2) / 65536."""
    units = np.arange(-(-n // 8), dtype=np.uint64)
    c = np.stack([units & np.uint64(0xffffffff), units >> np.uint64(32),
                  np.full_like(units, tensor), np.full_like(units, which)], -1)
    w = _philox(c, (step & 0xffffffff, step >> 32))
    h = np.stack([w & np.uint64(0xffff), w >> np.uint64(16)], -1).reshape(-1)[:n]
    return (h.astype(np.float64) + 0.5) / 65536


def test_generator_known_answers():
    """The published vectors of Philox4x32-10."""
    c = lambda *x: np.array([x], dtype=np.uint64)  # noqa: E731
    f = 0xffffffff
    assert [hex(x) for x in _philox(c(0, 0, 0, 0), (0, 0))[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    assert [hex(x) for x in _philox(c(f, f, f, f), (f, f))[0]] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


def test_refusals_of_roundings(lib):
    e = (G.gmm_adamw_tensor * 1)(G.gmm_adamw_tensor(param=256, grad=256, m=256, v=256, m_scale=256, v_scale=256, n=8))
    for r in (-1, 2):
        o = G.gmm_adamw_opts(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, step=1, state_bits=8, rounding=r)
        assert lib.gmm_adamw_step(e, 1, ctypes.byref(o), None) == G.GMM_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,capturable", [([300_001], False), ([256 * 40, 7, 1000], False), ([5000, 3000], True)])
@pytest.mark.parametrize("scale_of_gradients", [1.0, 1e-20])
def test_seeded_codes_are_those_of_the_rule(cuda, sizes, capturable, scale_of_gradients):
    """Each code is c or c + 1, c^2 <= value / S < (c + 1)^2, by u < p.  The new
    moments are the documented fp32 operations (numpy's float32 ones); p follows
    from them in 64 bits.  The kernel's p is off by at most 2^-24 x + 3 roundings
    of c^2 over 2 c + 1 for m (below 127 2^-23) and by the near root's 2^-22 of
    x, twice for its square, over 4 c^3 / c^4 and as many roundings for v (below
    255 2^-21): 2e-4 covers both, and closer ones may fall either way."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    f, near = np.float32, 2e-4
    rng = np.random.default_rng(sum(sizes))
    p = [torch.zeros(n, device="cuda") for n in sizes]
    opt = AdamW(p, betas=(0.9, 0.999), weight_decay=0.0, state_bits=8, rounding="seeded", capturable=capturable,
                step=2 ** 33 + 5)
    for step in range(2 ** 33 + 6, 2 ** 33 + 10):
        gs = [(scale_of_gradients * rng.standard_normal(n) * np.exp(2 * rng.standard_normal(n))).astype(f) for n in sizes]
        held = [[opt.state[k][i].cpu().numpy().astype(f) for k in ("m", "v", "m_scale", "v_scale")] for i in range(len(sizes))]
        opt.step([torch.from_numpy(g).cuda() for g in gs])
        for i, (n, g) in enumerate(zip(sizes, gs)):
            per = lambda s: np.repeat(s, 256)[:n]  # noqa: E731
            m, v, ms, vs = held[i]
            m, r = m * np.abs(m) * per(ms), v * v * per(vs)
            m = m * f(0.9) + g * f(1 - 0.9)
            v = (r * r) * f(0.999) + (g * g) * f(1 - 0.999)
            for x, top, which, name in ((m, 127, 0, "m"), (np.sqrt(v), 255, 1, "v")):
                big = np.array([np.abs(x[j:j + 256]).max() for j in range(0, n, 256)])
                scale = big * f(1.0 / (top * top))
                assert np.array_equal(opt.state[name + "_scale"][i].cpu().numpy(), scale)
                y = (np.abs(x) * per((f(1) / big) * f(top * top))).astype(np.float64)
                c = np.floor(np.sqrt(y))
                prob = (y - c * c) / (2 * c + 1) if which == 0 else (y ** 2 - c ** 4) / ((c + 1) ** 4 - c ** 4)
                u = _uniform(n, step, i, which)
                want = np.minimum(c + (u < prob), top)
                got = np.abs(opt.state[name][i].cpu().numpy().astype(np.float64))
                if which == 1:
                    want = np.where(x > 0, np.maximum(want, 1), want)
                else:
                    sign = np.sign(opt.state[name][i].cpu().numpy().astype(f))
                    assert ((sign == np.sign(x)) | (sign == 0)).all()
                off = got != want
                assert not (off & (np.abs(u - prob) > near)).any(), (step, name, np.flatnonzero(off & (np.abs(u - prob) > near))[:5])
                assert (np.abs(got - want) <= 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("value", [0.3, 0.011, 1e-4])
def test_seeded_codes_are_unbiased(cuda, value):
    """One step from zero of n equal gradients beside each block's largest: the
    mean of what is held is the value, up to six standard deviations of the mean
    of n independent choices between two neighbours (half their distance each)."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    blocks = 4000
    g = torch.full((blocks, 256), value, device="cuda")
    g[:, 0] = 1.0
    p = torch.zeros(blocks * 256, device="cuda")
    opt = AdamW([p], state_bits=8, rounding="seeded")
    opt.step([g.reshape(-1)])
    m, v = (t[0].double().reshape(blocks, 256)[:, 1:] for t in opt.moments())
    n = m.numel()
    for got, want, top, power in ((m, 0.1 * value, 127, 1), (v, 0.001 * value ** 2, 255, 2)):
        c = int(top * value ** 0.5)  # root of (value / largest) x top^2
        unit = (0.1 / 127 ** 2) if power == 1 else 0.001 ** 0.5 / 255 ** 2
        gap = ((c + 1) ** 2 * unit) ** power - (c ** 2 * unit) ** power
        assert c > 0 and abs(float(got.mean()) - want) <= 6 * gap / 2 / n ** 0.5 + 1e-5 * want


@pytest.mark.gpu
@pytest.mark.parametrize("later", [0.01, 0.0])
def test_averages_fall_again(cuda, later):
    """Half of every block's gradients shrink, or end, after 1000 of 10000 steps.
    v held in 8 bits follows the average in fp32: a code's steps are a walk with
    p (1 - p) near 0.00025 c a step over some 500 steps, a relative deviation of
    v of about 1.4 / sqrt(c), 0.3 at c = 25, so the mean of 2048 independent ones
    deviates by 0.7 %: 10 % is fourteen of these.  Where the gradients end m is
    zero (0.9^9000 of a code of 127^2 is no chance) and the parameters rest."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n = 4096
    p, q = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    a = AdamW([p], weight_decay=0.0, state_bits=8, rounding="seeded")
    b = AdamW([q], weight_decay=0.0)
    half = torch.arange(n, device="cuda") % 2 == 0
    for t in range(10000):
        x = torch.randn(n, device="cuda", generator=g)
        if t >= 1000:
            x = torch.where(half, x * later, x)
        a.step([x])
        b.step([x])
        if t == 6000:
            at = p.clone()
    (m8,), (v8,) = a.moments()
    (_,), (v,) = b.moments()
    # v's smallest code holds (max root / 255^2)^2 whatever the average
    least = (v.max().sqrt() / 255 ** 2) ** 2
    for part in (half, ~half):
        want = v[part].double().mean()
        assert abs(v8[part].double().mean() - want) <= 0.1 * want + 2 * least
    if later == 0:
        assert not m8[half].any()
        assert torch.equal(p[half], at[half])


@pytest.mark.gpu
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("grad", ["float32", "bfloat16"])
def test_seeded_steps_repeat_and_resume(cuda, grad, master):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    p0 = [torch.randn(k, device="cuda", generator=g).bfloat16() for k in (3000, 700)]
    grads = [[torch.randn(k, device="cuda", generator=g).to(getattr(torch, grad)) for k in (3000, 700)] for _ in range(4)]

    def run(stop=4, p=None, **kw):
        p = [t.clone() for t in p0] if p is None else p
        opt = AdamW(p, state_bits=8, rounding="seeded", master=master, **kw)
        for x in grads[opt.steps:stop]:
            opt.step(x)
        return p, opt

    p, one = run()
    q, two = run(capturable=True)
    h, half = run(stop=2)
    h, rest = run(p=h, step=half.steps, state={k: [t.clone() for t in ts] for k, ts in half.state.items()})
    for k in ("m", "v", "m_scale", "v_scale"):
        for x, y, z in zip(one.state[k], two.state[k], rest.state[k]):
            assert torch.equal(x, y) and torch.equal(x, z), k
    for x, z in zip(p, h):
        assert torch.equal(x, z)
    assert not torch.equal(one.state["m"][0][:700], one.state["m"][1])


@pytest.mark.gpu
def test_rounding_of_8_bits_is_asked_for(cuda):
    import torch
    import warnings
    from soft_clustering_gb300.adamw import AdamW
    p = [torch.zeros(8, device="cuda")]
    with pytest.raises(ValueError):
        AdamW(p, state_bits=8, rounding="up")
    with pytest.warns(UserWarning, match="seeded"):
        AdamW(p, state_bits=8)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        AdamW(p, state_bits=8, rounding="nearest")
        AdamW(p, state_bits=8, rounding="seeded")
        AdamW(p)


# ---------------------------------------------- values at the ends of the range

def _step32(held, g, n, b1=0.9, b2=0.999):
    """The new fp32 moments (m, v) from 8-bit state, each operation rounded once."""
    f = np.float32
    m, v, ms, vs = held
    per = lambda s: np.repeat(s, 256)[:n]  # noqa: E731
    m, r = m * np.abs(m) * per(ms), v * v * per(vs)
    return m * f(b1) + g * f(1 - b1), (r * r) * f(b2) + (g * g) * f(1 - b2)


TINY = [1e-17, 1e-18, 1e-19, 4e-20, 1e-20, 3e-21, 1e-21, 1e-22, 1e-25, 1e-29, 1e-36]


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [0.0, 1e-12, 1e-10, 1e-8])
@pytest.mark.parametrize("beside", [0.0, 1e-15, 1.0])
def test_small_values_in_8_bits(cuda, eps, beside):
    """Gradients whose v is subnormal or nearly so, alone in a block and beside
    larger ones: scales and codes are those of the documented fp32 operations,
    and the update is the formula's of those moments in 64 bits.  Its error: the
    near root and reciprocal 2^-23 each, the roundings of the two corrections,
    eps, two products and a sum 2^-24 each: 10 x 2^-24 of the update, and 2^-24
    of the parameter for each of decay, its product and the difference."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    f, lr, wd = np.float32, 0.01, 0.1
    rng = np.random.default_rng(int(beside) + 1)
    n = 256 * len(TINY) + 77
    size = np.concatenate([np.repeat(TINY, 256), np.full(77, 1e-20)])
    p = torch.from_numpy(rng.standard_normal(n).astype(f)).cuda()
    opt = AdamW([p], lr=lr, betas=(0.9, 0.999), eps=eps, weight_decay=wd, state_bits=8, rounding="nearest")
    with np.errstate(all="ignore"):
        for step in range(1, 4):
            g = (size * np.sign(rng.standard_normal(n)) * (1 + rng.random(n))).astype(f)
            if beside:
                g[::64] = beside
            held = [opt.state[k][0].cpu().numpy().astype(f) for k in ("m", "v", "m_scale", "v_scale")]
            before = p.double().cpu().numpy()
            opt.step([torch.from_numpy(g).cuda()])
            m, v = _step32(held, g, n)
            root = np.sqrt(v)
            for x, top, name in ((m, 127, "m"), (root, 255, "v")):
                big = np.array([np.abs(x[j:j + 256]).max() for j in range(0, n, 256)])
                scale = np.where(big >= f(1e-30), big * f(1.0 / (top * top)), f(0))
                assert np.array_equal(opt.state[name + "_scale"][0].cpu().numpy(), scale), (step, name)
                inv = np.where(scale > 0, (f(1) / big) * f(top * top), f(0)).astype(f)
                c = np.rint(np.sqrt(np.abs(x) * np.repeat(inv, 256)[:n]))
                c = np.where((x > 0) & (c < 1), f(1), c) if name == "v" else c * np.sign(x)
                got = opt.state[name][0].cpu().numpy().astype(f)
                assert np.array_equal(got, c), (step, name, np.flatnonzero(got != c)[:5])
            with np.errstate(all="ignore"):
                m, v = m.astype(np.float64), v.astype(np.float64)
                up = lr / (1 - 0.9 ** step) * m / (np.sqrt(v) / np.sqrt(1 - 0.999 ** step) + eps)
            ok = (v > 0) | (eps > 0)  # elsewhere the formula divides by zero
            after = before * (1 - lr * wd) - up
            bound = 1.01 * 2.0 ** -24 * (10 * np.abs(up) + 3 * (np.abs(before) + np.abs(up)))
            off = np.abs(p.double().cpu().numpy() - after)
            assert (off[ok] <= bound[ok]).all(), (step, size[ok][(off[ok] - bound[ok]).argmax()])
            p[torch.from_numpy(~ok).cuda()] = 1.0  # infinite there, as the formula says


def test_tensors_with_memory_in_common_are_refused():
    """One launch would write them twice, in no order."""
    import torch
    from soft_clustering_gb300.adamw import _apart
    x = torch.zeros(100)
    _apart([("a", x[:50]), ("b", x[50:]), ("c", None), ("d", x[:0]), ("e", torch.zeros(3))])
    _apart([])
    for a, b in ((x, x), (x[:51], x[50:]), (x, x[10:20]), (x[99:], x)):
        with pytest.raises(ValueError, match="memory in common"):
            _apart([("a", a), ("x", torch.zeros(4)), ("b", b)])


@pytest.mark.gpu
def test_a_parameter_given_twice_is_refused(cuda):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    p = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError, match="memory in common"):
        AdamW([p, p[90:]])
    opt = AdamW([p, torch.zeros(100, device="cuda")])
    opt.state["v"][1] = opt.state["m"][0]
    with pytest.raises(ValueError, match="memory in common"):
        opt.step([p, p])
    assert not p.any() and opt.steps == 0


@pytest.mark.gpu
def test_gradients_that_are_refused(cuda):
    """Anything but a dense tensor of the parameter's size on its device, first
    or last in the list; nothing is changed."""
    import torch
    p, grads, opt = _make()
    kept = [t.clone() for t in p]
    for at in (0, 1):
        n = p[at].numel()
        for bad in (None, 3, np.zeros(n, np.float32), torch.zeros(n), torch.zeros(n + 1, device="cuda"),
                    torch.zeros(2 * n, device="cuda")[::2], torch.zeros(n, device="cuda", dtype=torch.int32),
                    torch.zeros(n, device="cuda", dtype=torch.float64)):
            g = list(grads[0])
            g[at] = bad
            with pytest.raises(ValueError, match="grads.%d" % at):
                opt.step(g)
    assert opt.steps == 0
    for a, b in zip(p, kept):
        assert torch.equal(a, b)
