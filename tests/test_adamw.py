"""AdamW over many tensors (gmm_adamw_step, gmm_adamw_moments, AdamW).

The reference is the formula in 64 bits.  Tolerances, from the operations
alone (u = 2^-24; first order, times 1.01):
  m       3 u (|b1 m| + |c1 g|) plus the roundings of b1 and 1 - b1: 5 u
  v       4 u and the same: 6 u of the sum (all terms positive)
  update  m's error and that of sqrt(v), 2 products, a sum, a division: with
          relative error of m up to 5 u (|b1 m| + |c1 g|) / |m|
  p       u |p| x 3 plus the update's error, plus the type's rounding
8-bit moments: |sqrt(x / S) - c| <= 1/2 up to fp32 rounding, so
|x - c^2 S| <= (c + 1/4) S, widened by 1e-5 (c + 1)^2 S for the fp32 steps.
"""
import math

import numpy as np
import pytest

import soft_clustering_gb300 as G

U = 2.0 ** -24
UT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUB = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
LR, B1, B2, EPS, WD = 1e-2, 0.9, 0.999, 1e-8, 0.1


def _dt(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


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


def test_refusals(lib):
    import ctypes
    ok = dict(param=256, grad=256, m=256, v=256, n=8)
    opts = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, step=1, state_bits=32)

    def call(t=None, o=None, count=1):
        e = (G.gmm_adamw_tensor * 1)(G.gmm_adamw_tensor(**{**ok, **(t or {})}))
        op = G.gmm_adamw_opts(**{**opts, **(o or {})})
        return lib.gmm_adamw_step(e, count, ctypes.byref(op), None)

    bad = G.GMM_ERR_INVALID_ARG
    assert lib.gmm_adamw_step(None, 1, ctypes.byref(G.gmm_adamw_opts(**opts)), None) == bad
    assert lib.gmm_adamw_step(None, 0, None, None) == bad
    assert call(count=-1) == bad
    for t in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1),
              dict(param_dtype=3), dict(grad_dtype=-1), dict(param=258), dict(grad=1), dict(m=2),
              dict(master=2)):
        assert call(t) == bad, t
    for o in (dict(step=0), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1e-8),
              dict(lr=math.inf), dict(weight_decay=math.nan), dict(grad_scale=math.nan),
              dict(state_bits=16), dict(skip=2)):
        assert call(None, o) == bad, o
    assert call(None, dict(state_bits=8)) == bad  # no scales
    assert call(count=0) == G.GMM_OK
    assert call(dict(n=0, param=None, grad=None)) == G.GMM_OK  # an empty tensor


def _ref(p, g, m, v, t, gs=1.0):
    g = g * gs
    m2, v2 = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
    mag = np.abs(B1 * m) + np.abs((1 - B1) * g)
    den = np.sqrt(v2 / (1 - B2 ** t)) + EPS
    rate = LR / (1 - B1 ** t)
    p2 = p * (1 - LR * WD) - rate * m2 / den
    up = np.abs(rate * m2 / den)
    bm = 1.01 * 5 * U * mag
    bv = 1.01 * 6 * U * v2
    bp = 1.01 * (3 * U * np.abs(p) + rate * bm / den + 10 * U * up + U * np.abs(p2))
    return p2, m2, v2, bp, bm, bv


def _decoded(c, s, n):
    c = c.double().cpu().numpy()
    return np.sign(c) * c * c * np.repeat(s.double().cpu().numpy(), 256)[:n]


SIZES = [[1], [7], [256], [255, 257, 8], [1000, 1, 33, 0, 4096], [5000] * 3 + [300007]]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                          ("f16", "f32", False), ("f16", "f16", True), ("bf16", "bf16", True)])
@pytest.mark.parametrize("sizes", SIZES)
def test_step(cuda, bits, pt, gt, master, sizes):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    rng = np.random.default_rng(sum(sizes) + bits)
    t = lambda n, dt, s: torch.from_numpy((rng.standard_normal(n) * s).astype(np.float32)).to(_dt(dt)).cuda()  # noqa: E731
    params = [t(n, pt, 0.5) for n in sizes]
    opt = AdamW(params, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, state_bits=bits, master=master)
    for step in range(1, 4):
        grads = [t(n, gt, 0.1 * 10.0 ** (step - 2)) for n in sizes]
        for g in grads:  # a gradient of nothing, and one far larger than the rest
            if g.numel() > 2:
                g[0], g[1] = 0.0, 30.0
        before = []
        for i, n in enumerate(sizes):
            src = opt.state["master"][i] if master and opt.state["master"][i] is not None else params[i]
            if bits == 32:
                m, v = (opt.state[k][i].double().cpu().numpy() for k in "mv")
            else:
                m = _decoded(opt.state["m"][i], opt.state["m_scale"][i], n)
                v = _decoded(opt.state["v"][i], opt.state["v_scale"][i], n) ** 2
            before.append((src.double().cpu().numpy(), m, v))
        opt.step(grads, grad_scale=0.5)
        mo, vo = opt.moments()
        for i, n in enumerate(sizes):
            p2, m2, v2, bp, bm, bv = _ref(before[i][0], grads[i].double().cpu().numpy(), *before[i][1:], step, 0.5)
            # 8 bits: the old moments come through c|c| S (2 roundings) and a square (2 more)
            bm, bv, bp = (bm * 2, bv * 2, bp * 2) if bits == 8 else (bm, bv, bp)
            got = params[i].double().cpu().numpy()
            if master and pt != "f32":
                ms = opt.state["master"][i].double().cpu().numpy()
                assert (np.abs(ms - p2) <= bp).all()
                assert torch.equal(opt.state["master"][i].to(_dt(pt)), params[i])
            assert (np.abs(got - p2) <= bp + (UT[pt] + U) * (np.abs(p2) + bp) + SUB[pt]).all()
            gm, gv = mo[i].double().cpu().numpy(), vo[i].double().cpu().numpy()
            if bits == 32:
                assert (np.abs(gm - m2) <= bm).all() and (np.abs(gv - v2) <= bv).all()
            else:
                sm = np.repeat(opt.state["m_scale"][i].double().cpu().numpy(), 256)[:n]
                sv = np.repeat(opt.state["v_scale"][i].double().cpu().numpy(), 256)[:n]
                cm = np.abs(opt.state["m"][i].double().cpu().numpy())
                cv = opt.state["v"][i].double().cpu().numpy()
                r2 = np.sqrt(v2)
                assert (np.abs(gm - m2) <= (cm + 0.25) * sm + 1e-5 * (cm + 1) ** 2 * sm + bm).all()
                near = np.abs(np.sqrt(gv) - r2) <= (cv + 0.25) * sv + 1e-5 * (cv + 1) ** 2 * sv
                assert (near | ((cv == 1) & (r2 <= sv))).all()  # a positive value keeps a code above zero
                assert ((cv > 0) == (r2 > 0)).all()
                if n:
                    assert cm.max() == 127 and cv.max() == 255


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 4, 8])
def test_views_at_odd_addresses_give_the_same(cuda, bits, shift):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    rng = np.random.default_rng(shift)
    n = 1337
    p0, g0 = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(2))
    out = []
    for s in (0, shift):
        p, g = (torch.zeros(n + s, dtype=torch.bfloat16, device="cuda")[s:].copy_(x) for x in (p0, g0))
        opt = AdamW([p], state_bits=bits, lr=LR)
        opt.step([g])
        opt.step([g])
        out.append([p, *opt.state["m"], *opt.state["v"]])
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_more_tensors_than_a_launch_holds(cuda):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    n = [1 + (7 * i) % 500 for i in range(1000)]
    params = [torch.full((k,), 1.0, device="cuda") for k in n]
    grads = [torch.full((k,), 0.01 * (1 + i % 5), device="cuda") for i, k in enumerate(n)]
    AdamW(params, lr=0.5, weight_decay=0.0).step(grads)
    # the first step moves every element by lr, up to eps and rounding
    for p in params:
        assert ((p - 0.5).abs() <= 1e-5).all()


@pytest.mark.gpu
def test_skip_changes_nothing(cuda):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    for bits in (32, 8):
        p = torch.randn(1000, device="cuda")
        opt = AdamW([p], state_bits=bits)
        opt.step([torch.randn_like(p)])
        kept = [x.clone() for x in (p, opt.state["m"][0], opt.state["v"][0])]
        opt.step([torch.full_like(p, float("nan"))], skip=torch.ones(1, dtype=torch.int32, device="cuda"))
        for a, b in zip(kept, (p, opt.state["m"][0], opt.state["v"][0])):
            assert torch.equal(a, b)
        opt.step([torch.randn_like(p)], skip=torch.zeros(1, dtype=torch.int32, device="cuda"))
        assert not torch.equal(kept[0], p) and torch.isfinite(p).all()


@pytest.mark.gpu
def test_resume_continues_bit_for_bit(cuda):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    for bits in (32, 8):
        torch.manual_seed(3)
        a = [torch.randn(n, device="cuda").bfloat16() for n in (300, 5000)]
        gs = [[torch.randn_like(p) for p in a] for _ in range(4)]
        one = AdamW(a, state_bits=bits, master=True)
        one.step(gs[0])
        one.step(gs[1])
        b = [p.clone() for p in a]
        two = AdamW(b, state_bits=bits, master=True, step=one.steps,
                    state={k: [x.clone() for x in v] for k, v in one.state.items()})
        for g in gs[2:]:
            one.step(g)
            two.step(g)
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_tiny_and_zero_blocks(cuda):
    """Blocks of zeros and of values below the smallest scale stay finite."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    p = torch.ones(1024, device="cuda")
    g = torch.zeros(1024, device="cuda")
    g[256:512] = 1e-25
    g[512:768] = 1e-36
    opt = AdamW([p], state_bits=8, weight_decay=0.0)
    for _ in range(3):
        opt.step([g])
    assert torch.isfinite(p).all() and (p[:256] == 1).all()
    m, v = opt.moments()
    assert torch.isfinite(m[0]).all() and torch.isfinite(v[0]).all()


@pytest.mark.gpu
def test_python_refusals(cuda):
    import torch
    from soft_clustering_gb300.adamw import AdamW
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4)])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4, device="cuda", dtype=torch.float64)])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4, 4, device="cuda").t()[:, 1:]])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4, device="cuda")], state_bits=4)
    opt = AdamW([torch.zeros(4, device="cuda")])
    with pytest.raises(ValueError):
        opt.step([])
    with pytest.raises(ValueError):
        opt.step([torch.zeros(5, device="cuda")])
    with pytest.raises(ValueError):
        opt.step([torch.zeros(8, device="cuda")[::2]])
    with pytest.raises(G.GmmError):
        opt.lr = float("nan")
        opt.step([torch.zeros(4, device="cuda")])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [256 * 40, 300_001])
def test_codes_are_those_of_exact_roots(cuda, n):
    """8-bit codes and scales equal the documented fp32 operations, each
    rounded once (numpy's float32 operations are), over several steps."""
    import torch
    from soft_clustering_gb300.adamw import AdamW
    f = np.float32
    rng = np.random.default_rng(n)
    p = torch.zeros(n, device="cuda")
    opt = AdamW([p], lr=1e-3, betas=(B1, B2), eps=EPS, weight_decay=0.0, state_bits=8)
    blocks = -(-n // 256)
    pad = lambda x: np.concatenate([x, np.zeros(blocks * 256 - n, f)]).reshape(blocks, 256)  # noqa: E731
    m, r = np.zeros((blocks, 256), f), np.zeros((blocks, 256), f)
    for step in range(4):
        g = (rng.standard_normal(n) * np.exp(2 * rng.standard_normal(n))).astype(f)
        opt.step([torch.from_numpy(g).cuda()])
        g = pad(g)
        m = m * f(B1) + g * f(1 - B1)
        v = (r * r) * f(B2) + (g * g) * f(1 - B2)
        root = np.sqrt(v)
        for x, top, name in ((m, 127, "m"), (root, 255, "v")):
            big = np.abs(x).max(1)
            scale = big * f(1.0 / (top * top))
            inv = np.where(big > 0, (f(1) / np.where(big > 0, big, f(1))) * f(top * top), f(0)).astype(f)
            c = np.rint(np.sqrt(np.abs(x) * inv[:, None]))
            c = np.where((x > 0) & (c < 1), f(1), c) if name == "v" else c * np.sign(x)
            assert np.array_equal(opt.state[name + "_scale"][0].cpu().numpy(), scale), (step, name)
            got = opt.state[name][0].cpu().numpy().astype(f)
            assert np.array_equal(got, c.reshape(-1)[:n]), (step, name, (got != c.reshape(-1)[:n]).sum())
            val = c * np.abs(c) * scale[:, None]
            if name == "m":
                m = val
            else:
                r = val
