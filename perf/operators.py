"""Cases and plain forms of the local-expert operators.

A fitted mixture answers with each point's top-m components and their
responsibilities (ids, gamma).  Behind that gate stand local experts: a
point's row goes to its components (route and spread), each component
multiplies its rows by its own weights (product), the answers come back
summed with gamma (collect), and the weights are learnt by AdamW.

  route    ids [N, m] -> offsets [K+1], entry, slot, and the rows in order;
           backward: the gradient of the rows, summed back per point
  combine  forward:  out[n] = sum_t gamma[n, t] Z[slot[n, t]]
           backward: dZ[slot[n, t]] = gamma[n, t] dout[n],
                     dgamma[n, t] = <dout[n], Z[slot[n, t]]>
  product  forward:  Y[r] = W_k A[r] for the rows r of expert k
           backward: dA[r] = W_k^T dY[r],  dW_k = sum_r dY[r] A[r]^T
  adamw    one step over a list of tensors, moments in 32 or 8 bits

``run`` computes them with elementary torch operations in 32 bits, or, with
``own`` set, through soft_clustering_gb300.
"""
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256  # elements that share one scale of an 8-bit moment
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one query against an index of 4096 lists: latency alone
        dict(name="route one query", op="route", direction="forward", N=1, m=4, K=4096, D=128, dtype="f16", drop=0.0),
        # the gradient that comes back to a batch of wide rows
        dict(name="route batch, gradient", op="route", direction="backward", N=16385, m=2, K=64, D=1024, dtype="bf16", drop=0.0),
        # embeddings put in order of their lists, entries below the responsibility threshold left out
        dict(name="route embeddings", op="route", direction="forward", N=2000003, m=4, K=4096, D=128, dtype="f16", drop=0.3),
        # a handful of queries' answers
        dict(name="combine few", op="combine", direction="forward", N=5, m=4, K=64, D=2048, dtype="bf16", drop=0.0),
        # a training batch's answers
        dict(name="combine batch", op="combine", direction="forward", N=65536, m=2, K=64, D=2048, dtype="bf16", drop=0.0),
        # gradients of embeddings' answers and of their responsibilities
        dict(name="combine embeddings, gradient", op="combine", direction="backward", N=1000003, m=4, K=256, D=128, dtype="f16", drop=0.2),
        # eight queries with two experts each: few rows, every weight read once
        dict(name="product few", op="product", direction="forward", rows=16, K=64, d_in=1024, d_out=2048, dtype="bf16"),
        # embeddings through small experts: rows read and written
        dict(name="product embeddings", op="product", direction="forward", rows=1000001, K=256, d_in=128, d_out=128, dtype="f16"),
        # a large batch through wide experts: arithmetic
        dict(name="product batch", op="product", direction="forward", rows=65536, K=32, d_in=2048, d_out=2048, dtype="bf16"),
        # the two gradients of a training batch of a ragged size
        dict(name="product batch, gradients", op="product", direction="backward", rows=16385, K=64, d_in=1024, d_out=2048, dtype="bf16"),
        # the parameters of a small mixture: weights, means, variances
        dict(name="adamw small", op="adamw", tensors=3, total=1160, dtype="f32", bits=32),
        # a layer of experts with many tensors of ragged sizes, moments in 8 bits
        dict(name="adamw 8-bit", op="adamw", tensors=120, total=200000000, dtype="bf16", bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "combine", "product", "adamw"])
    if op in ("route", "combine"):
        direction = rng.choice(["forward", "backward"])
        D = rng.choice([64, 128, 256, 512, 1024, 2048, 8 * _log(rng, 2, 256), _log(rng, 8, 2048)])
        m = rng.choice([1, 2, 3, 4, 8])
        dtype = rng.choice(["f16", "bf16", "f32"])
        most = min(2000003, 500000000 // (D * m))
        return dict(op=op, direction=direction, N=_log(rng, 1, most), m=m, K=_log(rng, 8, 4096), D=D, dtype=dtype,
                    drop=rng.choice([0.0, 0.1, 0.5]))
    if op == "product":
        direction = rng.choice(["forward", "backward"])
        d_in, d_out = (rng.choice([64, 128, 256, 512, 1024, 2048, 8 * _log(rng, 8, 256)]) for _ in range(2))
        K = _log(rng, 8, min(256, 200000000 // (d_in * d_out)))
        most = min(1000001, 250000000000 // (2 * d_in * d_out), 300000000 // (d_in + d_out))
        return dict(op=op, direction=direction, rows=_log(rng, 1, most), K=K, d_in=d_in, d_out=d_out,
                    dtype=rng.choice(["f16", "bf16"]))
    bits = rng.choice([8, 32])
    tensors = _log(rng, 1, 200)
    return dict(op="adamw", tensors=tensors, total=_log(rng, 40 * tensors, 100000000), dtype=rng.choice(["f32", "bf16", "f16"]), bits=bits)


def _sizes(case):
    """Element counts of the list's tensors, ragged, `total` in all (the same for every seed)."""
    r = random.Random(case["tensors"] * 7919 + case["total"])
    w = [0.05 + r.random() ** 3 for _ in range(case["tensors"])]
    sizes = [max(1, int(case["total"] * x / sum(w))) for x in w]
    sizes[-1] += max(0, case["total"] - sum(sizes))
    return sizes


# ----------------------------------------------------------------- inputs

def _popularity(K, g):
    """How often each expert is the best one: uneven, as mixture weights are."""
    return torch.softmax(0.5 * torch.randn(K, device="cuda", generator=g), 0)


def _assignment(case, g):
    """Top-m ids (distinct per point, -1 where the entry is left out) and descending gammas."""
    N, m, K = case["N"], case["m"], case["K"]
    first = torch.multinomial(_popularity(K, g), N, replacement=True, generator=g)
    step = 1 + torch.randint(0, max(1, K // m), (N, m - 1), device="cuda", generator=g)
    rest = torch.cumsum(step, 1)
    ids = torch.cat([first[:, None], (first[:, None] + rest) % K], 1).to(torch.int32)
    gamma = torch.softmax(2.0 * torch.randn(N, m, device="cuda", generator=g), 1).sort(1, descending=True)[0].contiguous()
    if case["drop"] > 0:
        out = torch.rand(N, m, device="cuda", generator=g) < case["drop"]
        out[:, 0] &= torch.rand(N, device="cuda", generator=g) < 0.02  # a few points keep none of the first
        ids = torch.where(out, torch.full_like(ids, -1), ids)
    return ids.contiguous(), gamma


def _plan(ids, K):
    """offsets [K+1] int64, entry [N m] int32 (-1 past the kept ones), slot [N, m] int32 (-1: left out)."""
    flat = ids.reshape(-1).long()
    E = flat.numel()
    key = torch.where((flat >= 0) & (flat < K), flat, torch.full_like(flat, K))
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(K + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), torch.cumsum(counts[:K], 0)])
    pos = torch.arange(E, device=ids.device)
    entry = torch.where(pos < offsets[K], order, torch.full_like(order, -1)).to(torch.int32)
    slot = torch.empty_like(pos).scatter_(0, order, pos)
    slot = torch.where(key < K, slot, torch.full_like(slot, -1)).to(torch.int32)
    return offsets, entry, slot.reshape(ids.shape)


def _rand(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(case), "own": {}}
    if case["op"] in ("route", "combine"):
        dt, N, m, D = DT[case["dtype"]], case["N"], case["m"], case["D"]
        s["ids"], s["gamma"] = _assignment(case, g)
        back = case["direction"] == "backward"
        if case["op"] == "route" and not back:
            s["X"] = _rand((N, D), dt, g)
            return s
        s["offsets"], s["entry"], s["slot"] = _plan(s["ids"], case["K"])
        if case["op"] == "route":
            s["dY"] = _rand((N * m, D), dt, g, 0.01)
        else:
            s["Z"] = _rand((N * m, D), dt, g)
            if back:
                s["dout"] = _rand((N, D), dt, g, 0.01)
        return s
    if case["op"] == "product":
        dt, K, R = DT[case["dtype"]], case["K"], case["rows"]
        who = torch.multinomial(_popularity(K, g), R, replacement=True, generator=g)
        counts = torch.bincount(who, minlength=K)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(counts, 0)])
        s["most"] = int(counts.max())
        s["W"] = _rand((K, case["d_out"], case["d_in"]), dt, g, case["d_in"] ** -0.5)
        s["A"] = _rand((R, case["d_in"]), dt, g)
        if case["direction"] == "backward":
            s["dY"] = _rand((R, case["d_out"]), dt, g, 0.01)
        return s
    # adamw: the tensors are views of one buffer, each starting on a block
    dt, sizes = DT[case["dtype"]], _sizes(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += -(-n // BLOCK) * BLOCK
    live = torch.zeros(at, dtype=torch.bool, device="cuda")
    for o, n in zip(starts, sizes):
        live[o:o + n] = True
    live = live.float()
    s["starts"], s["sizes"], s["step"] = starts, sizes, 1000
    s["p"] = (torch.randn(at, device="cuda", generator=g) * 0.05 * live).to(dt)
    s["grad"] = (torch.randn(at, device="cuda", generator=g) * 0.01 * live).to(dt)
    # a layer's elements see gradients of very different size
    size = torch.exp(torch.randn(at, device="cuda", generator=g)) * 0.01 * live
    mom, root = torch.randn(at, device="cuda", generator=g) * 0.3 * size, size
    if case["bits"] == 32:
        s["m"], s["v"] = mom, root * root
    else:
        s["m"], s["ms"] = _encode(mom, 127)
        s["v"], s["vs"] = _encode(root, 255)
    return s


# ------------------------------------------------- 8-bit moments, plainly

def _encode(x, top):
    """Codes and scales of blocks of 256: x stands as c |c| S with S = max|x| / top^2; the root of x / S is rounded.
    A block whose largest value is below 1e-30 stands as zeros."""
    b = x.reshape(-1, BLOCK)
    big = b.abs().amax(1)
    big = torch.where(big >= 1e-30, big, torch.zeros_like(big))
    scale = big * (1.0 / (top * top))
    inv = torch.where(big > 0, torch.reciprocal(big) * float(top * top), torch.zeros_like(big))
    c = torch.round(torch.sqrt(b.abs() * inv[:, None])).clamp_(max=float(top))
    if top == 255:  # a positive value keeps a code above zero
        c = torch.where(b > 0, c.clamp(min=1.0), c)
        return c.to(torch.uint8).reshape(-1), scale
    return (c * torch.sign(b)).to(torch.int8).reshape(-1), scale


def _decode(c, scale):
    f = c.reshape(-1, BLOCK).float()
    return (f * f.abs() * scale[:, None]).reshape(-1)


# -------------------------------------------------------------------- run

def _padded(rows, offsets, K, most):
    """Each row's expert and place within it."""
    r = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets, r, right=True) - 1
    return e, r - offsets[e]


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        dt = DT[c["dtype"]]
        if c["direction"] == "backward":
            slot = s["slot"].long()
            rows = s["dY"].float()[slot.clamp(min=0)]
            return {"dX": (rows * (slot >= 0)[..., None]).sum(1).to(dt)}
        offsets, entry, slot = _plan(s["ids"], c["K"])
        rows = s["X"].float()[entry.long().clamp(min=0) // c["m"]]
        return {"offsets": offsets, "entry": entry, "slot": slot, "Y": (rows * (entry >= 0)[:, None]).to(dt)}
    if c["op"] == "combine":
        dt, slot = DT[c["dtype"]], s["slot"].long()
        kept = (slot >= 0)[..., None]
        rows = s["Z"].float()[slot.clamp(min=0)] * kept
        if c["direction"] == "forward":
            return {"out": (rows * s["gamma"][..., None]).sum(1).to(dt)}
        dout = s["dout"].float()
        dgamma = (rows * dout[:, None, :]).sum(2)
        n, t = s["entry"].long().clamp(min=0) // c["m"], s["entry"].long().clamp(min=0) % c["m"]
        w = s["gamma"][n, t] * (s["entry"] >= 0)
        return {"dZ": (dout[n] * w[:, None]).to(dt), "dgamma": dgamma}
    if c["op"] == "product":
        dt, K, R = DT[c["dtype"]], c["K"], c["rows"]
        e, at = _padded(R, s["offsets"], K, s["most"])
        W = s["W"].float()
        A = torch.zeros(K, s["most"], c["d_in"], device="cuda")
        A[e, at] = s["A"].float()
        if c["direction"] == "forward":
            return {"Y": torch.bmm(A, W.transpose(1, 2))[e, at].to(dt)}
        dY = torch.zeros(K, s["most"], c["d_out"], device="cuda")
        dY[e, at] = s["dY"].float()
        return {"dA": torch.bmm(dY, W)[e, at].to(dt), "dW": torch.bmm(dY.transpose(1, 2), A).to(dt)}
    s["step"] += 1
    t = s["step"]
    g = s["grad"].float()
    if c["bits"] == 32:
        mom, v = s["m"], s["v"]
    else:
        mom, root = _decode(s["m"], s["ms"]), _decode(s["v"], s["vs"])
        v = root * root
    mom = mom * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = torch.sqrt(v)
    den = root * ((1 - BETA2 ** t) ** -0.5) + EPS
    p = s["p"].float() * (1 - LR * DECAY) - (mom * (LR / (1 - BETA1 ** t))) / den
    s["p"].copy_(p.to(s["p"].dtype))
    if c["bits"] == 32:
        s["m"].copy_(mom)
        s["v"].copy_(v)
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    s["m"], s["ms"] = _encode(mom, 127)
    s["v"], s["vs"] = _encode(root, 255)
    root = _decode(s["v"], s["vs"])
    return {"p": s["p"], "m": _decode(s["m"], s["ms"]), "v": root * root}


def _own(s):
    import soft_clustering_gb300 as G

    c, h = s["case"], s["own"]
    if c["op"] in ("route", "combine"):
        x, N, m, D, K, dev = CODE[c["dtype"]], c["N"], c["m"], c["D"], c["K"], "cuda"
        if c["op"] == "route" and c["direction"] == "forward":
            from soft_clustering_gb300.experts import Router
            if not h:
                h["router"] = Router(N, m, K)
            r = h["router"]
            r.route(s["ids"])
            return {"offsets": r.offsets, "entry": r.entry, "slot": r.slot, "Y": r.spread(s["X"])}
        if c["op"] == "route":
            dX = torch.empty(N, D, dtype=s["dY"].dtype, device=dev)
            G.gmm_collect(s["dY"], x, N, D, m, N * m, s["slot"], None, dX)
            return {"dX": dX}
        if c["direction"] == "forward":
            out = torch.empty(N, D, dtype=s["Z"].dtype, device=dev)
            G.gmm_collect(s["Z"], x, N, D, m, N * m, s["slot"], s["gamma"], out)
            return {"out": out}
        dZ, dgamma = torch.empty_like(s["Z"]), torch.empty_like(s["gamma"])
        G.gmm_spread(s["dout"], x, N, D, m, K, N * m, s["slot"], s["offsets"], s["gamma"], s["Z"], dZ, dgamma)
        return {"dZ": dZ, "dgamma": dgamma}
    if c["op"] == "product":
        from soft_clustering_gb300.experts import ExpertProduct
        if not h:
            h["product"] = ExpertProduct(c["K"], c["d_in"], c["d_out"], DT[c["dtype"]], c["rows"])
        e = h["product"]
        if c["direction"] == "forward":
            return {"Y": e.forward(s["A"], s["offsets"], s["W"])}
        return {"dA": e.backward_rows(s["dY"], s["offsets"], s["W"]), "dW": e.backward_weights(s["dY"], s["A"], s["offsets"])}
    from soft_clustering_gb300.adamw import AdamW
    if not h:
        parts = lambda t, q=1: [t[o // q:-(-(o + n) // q)] for o, n in zip(s["starts"], s["sizes"])]  # noqa: E731
        state = {"m": parts(s["m"]), "v": parts(s["v"])}
        if c["bits"] == 8:
            state.update(m_scale=parts(s["ms"], BLOCK), v_scale=parts(s["vs"], BLOCK))
            h["m"], h["v"] = torch.zeros(len(s["p"]), device="cuda"), torch.zeros(len(s["p"]), device="cuda")
            h["out"] = parts(h["m"]), parts(h["v"])
        h["grads"] = parts(s["grad"])
        h["opt"] = AdamW(parts(s["p"]), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=c["bits"],
                         state=state, step=s["step"])
    h["opt"].step(h["grads"])
    if c["bits"] == 32:
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    h["opt"].moments(*h["out"])
    return {"p": s["p"], "m": h["m"], "v": h["v"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work

def work(case):
    if case["op"] in ("route", "combine"):
        N, m, K, D, es = case["N"], case["m"], case["K"], case["D"], SIZE[case["dtype"]]
        kept = N * m * (1 - case["drop"]) + (N * case["drop"] * 0.98 if case["drop"] else 0)  # the first entry mostly stays
        row = D * es
        if case["op"] == "route" and case["direction"] == "forward":
            return {"bytes": 12.0 * N * m + 8 * (K + 1) + N * row + N * m * row, "flops": 0.0}
        if case["op"] == "route":
            return {"bytes": 4.0 * N * m + kept * row + N * row, "flops": kept * D}
        if case["direction"] == "forward":
            return {"bytes": 8.0 * N * m + kept * row + N * row, "flops": 2.0 * kept * D}
        return {"bytes": 12.0 * N * m + kept * row + N * row + N * m * row, "flops": 3.0 * kept * D}
    if case["op"] == "product":
        R, K, i, o, es = case["rows"], case["K"], case["d_in"], case["d_out"], SIZE[case["dtype"]]
        used = K * (1 - (1 - 1 / K) ** R)  # experts with a row, about
        if case["direction"] == "forward":
            return {"bytes": es * (R * i + R * o + used * i * o) + 8.0 * (K + 1), "flops": 2.0 * R * i * o}
        return {"bytes": es * (2.0 * R * i + R * o + (used + K) * i * o) + 8.0 * (K + 1), "flops": 4.0 * R * i * o}
    n, es = case["total"], SIZE[case["dtype"]]
    per = 3 * es + 16 if case["bits"] == 32 else 3 * es + 4 + 16 / BLOCK + 8
    return {"bytes": float(n * per), "flops": 20.0 * n}


# ------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] in ("route", "combine"):
        N, m = case["N"], case["m"]
        if case["op"] == "route" and case["direction"] == "forward":
            flat = s["ids"].reshape(-1).long()
            kept = torch.nonzero((flat >= 0) & (flat < case["K"])).reshape(-1)
            first = kept[torch.argsort(flat[kept] * flat.numel() + kept)]
            Y = torch.zeros(N * m, case["D"], dtype=f, device="cuda")
            Y[:first.numel()] = s["X"].to(f)[torch.div(first, m, rounding_mode="floor")]
            return {"offsets": None, "entry": None, "slot": None, "Y": Y}
        src, w = (s["dY"], None) if case["op"] == "route" else (s["Z"], s["gamma"].to(f))
        out = torch.zeros(N, case["D"], dtype=f, device="cuda")
        if case["direction"] == "forward" or case["op"] == "route":
            for t in range(m):
                at = s["slot"][:, t].long()
                ok = torch.nonzero(at >= 0).reshape(-1)
                row = src[at[ok]].to(f)
                out[ok] += row if w is None else row * w[ok, t][:, None]
            return {"dX" if case["op"] == "route" else "out": out}
        dout = s["dout"].to(f)
        dZ, dgamma = torch.zeros(N * m, case["D"], dtype=f, device="cuda"), torch.zeros(N, m, dtype=f, device="cuda")
        for t in range(m):
            at = s["slot"][:, t].long()
            ok = torch.nonzero(at >= 0).reshape(-1)
            dgamma[ok, t] = torch.einsum("nd,nd->n", src[at[ok]].to(f), dout[ok])
            dZ[at[ok]] = dout[ok] * w[ok, t][:, None]
        return {"dZ": dZ, "dgamma": dgamma}
    if case["op"] == "product":
        o = s["offsets"].tolist()
        A, W = s["A"].to(f), s["W"]
        if case["direction"] == "forward":
            Y = torch.empty(case["rows"], case["d_out"], dtype=f, device="cuda")
            for k in range(case["K"]):
                Y[o[k]:o[k + 1]] = A[o[k]:o[k + 1]] @ W[k].to(f).T
            return {"Y": Y}
        dY, dA = s["dY"].to(f), torch.empty_like(A)
        dW = torch.zeros(W.shape, dtype=f, device="cuda")
        for k in range(case["K"]):
            a, b = o[k], o[k + 1]
            dA[a:b] = dY[a:b] @ W[k].to(f)
            dW[k] = dY[a:b].T @ A[a:b]
        return {"dA": dA, "dW": dW}
    # adamw, after one step
    t = s["step"] + 1
    bits = case["bits"]

    def value(c, scale):
        c = c.to(f)
        return torch.sign(c) * c ** 2 * scale.to(f).repeat_interleave(BLOCK)

    def kept(x, top, least):
        big = x.abs().reshape(-1, BLOCK).max(1).values.repeat_interleave(BLOCK)
        unit = torch.where(big > 0, big, torch.ones_like(big)) / top ** 2
        c = (x.abs() / unit).sqrt().round()
        c = torch.where(x.abs() > 0, c.clamp(min=least), c)
        return torch.sign(x) * c ** 2 * unit

    g, p = s["grad"].to(f), s["p"].to(f)
    mom = s["m"].to(f) if bits == 32 else value(s["m"], s["ms"])
    v = s["v"].to(f) if bits == 32 else value(s["v"], s["vs"]) ** 2
    mom = BETA1 * mom + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = p - LR * DECAY * p - LR * (mom / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    if bits == 32:
        return {"p": p, "m": mom, "v": v}
    return {"p": p, "m": kept(mom, 127, 0), "v": kept(v.sqrt(), 255, 1) ** 2}
