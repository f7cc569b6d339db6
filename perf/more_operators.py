"""Cases and plain forms of the learned gate's operators.

Local experts stand behind a gate.  The fitted mixture is one; a learned one
answers from logits L [N, K], a row for each point:

  gate     forward:  the m largest of a row (ids) and their share of
                     softmax(L) (gamma), and the row's log-sum-exp
           backward: the gradient of the logits from that of gamma
  balance  the same with what keeps components in use: entries of each
           component (counts), mass_k = sum_n p_nk, and
           loss = sum_k share_k mass_k with
           share_k = K counts_k / (sum counts * rows), rows those that count;
           backward adds coef * its gradient (share held fixed)
  distill  a teacher's top entries of each row (the mixture's top-m
           responsibilities, or a larger model's top logits) against the
           student's softmax(L / T):
           loss = scale T^2 sum_n w_n KL(q_n || p_n)
           forward: the loss; step: the loss and the gradient of the logits
  norm     layer norm of rows; backward: gradients of rows, weight and bias

``run`` computes them with elementary torch operations in 32 bits, or, with
``own`` set, through soft_clustering_gb300.
"""
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
COEF, EPS = 0.01, 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one query against the 4096 lists of an index: latency alone
        dict(name="gate one query", op="gate", direction="forward", N=1, K=4096, m=4, dtype="f16", normalised=False, drop=0.0, masked=0.0),
        # a batch of rows to two of 64 experts, weights that sum to one, some rows padding
        dict(name="gate batch", op="gate", direction="forward", N=65537, K=64, m=2, dtype="bf16", normalised=True, drop=0.1, masked=0.0),
        # the gradient of a batch's responsibilities over many components
        dict(name="gate wide, gradient", op="gate", direction="backward", N=65536, K=4096, m=4, dtype="bf16", normalised=False, drop=0.0, masked=0.0),
        # a handful of rows, eight components: a training loop's smallest step
        dict(name="balance small", op="balance", direction="forward", N=512, K=8, m=2, dtype="f32", normalised=False, drop=0.0, masked=0.0),
        # embeddings to four of 256 components, some of which are empty
        dict(name="balance embeddings", op="balance", direction="forward", N=1000003, K=256, m=4, dtype="f16", normalised=False, drop=0.0, masked=0.1),
        # a training batch's gradient with the balance loss in it
        dict(name="balance batch, gradient", op="balance", direction="backward", N=262144, K=1024, m=2, dtype="bf16", normalised=True, drop=0.1, masked=0.0),
        # seven rows of a vocabulary against a teacher's 64 top logits: an evaluation step
        dict(name="distill few", op="distill", direction="forward", N=7, K=131072, m=64, dtype="bf16", teacher="logits", T=1.0, drop=0.0),
        # a gate taught by the mixture's top-4 responsibilities, weighted rows
        dict(name="distill embeddings", op="distill", direction="step", N=1000003, K=256, m=4, dtype="f16", teacher="gamma", T=1.0, drop=0.1),
        # a vocabulary of an odd size, soft targets
        dict(name="distill vocabulary", op="distill", direction="step", N=8191, K=50257, m=32, dtype="bf16", teacher="logits", T=2.0, drop=0.0),
        # one row of a decoding step
        dict(name="norm one row", op="norm", direction="forward", N=1, D=1024, dtype="bf16", weights="bf16"),
        # embeddings
        dict(name="norm embeddings", op="norm", direction="forward", N=2000003, D=128, dtype="f16", weights="f32"),
        # the gradients of a training batch of wide rows
        dict(name="norm batch, gradients", op="norm", direction="backward", N=65536, D=4096, dtype="bf16", weights="bf16"),
    ]


def scale_of(case):
    """A loss is a mean over the rows, or with fp16 gradients (of which a mean's would be subnormal) a sum, scaled back by the optimiser."""
    return 1.0 if case["dtype"] == "f16" else 1.0 / case["N"]


def coef_of(case):
    """The balance loss is of the size of one, so its gradient is a mean's."""
    return COEF * case["N"] * scale_of(case)


MOST = 500000000  # bytes of a drawn case's logits or rows


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _size(rng, lo, hi):
    """A width: a power of two, a multiple of eight, or any."""
    n = _log(rng, lo, hi)
    kind = rng.choice(["power", "eight", "any"])
    if kind == "power":
        return min(hi, 1 << (n.bit_length() - 1))
    return min(hi, max(lo, n // 8 * 8)) if kind == "eight" and n >= 8 else n


def draw(rng):
    op = rng.choice(["gate", "balance", "distill", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        D = _size(rng, 2, 16384)
        return dict(op=op, direction=rng.choice(["forward", "backward"]), N=_log(rng, 1, min(2000003, MOST // (D * SIZE[dtype]))), D=D,
                    dtype=dtype, weights=rng.choice([dtype, "f32"]))
    if op == "distill":
        K = _size(rng, 2, 131072)
        N = _log(rng, 1, min(1000003, MOST // (K * SIZE[dtype])))
        return dict(op=op, direction=rng.choice(["forward", "step"]), N=N, K=K, m=min(K, _log(rng, 1, 64)), dtype=dtype,
                    teacher=rng.choice(["gamma", "logits"]), T=rng.choice([1.0, 2.0, 0.5]), drop=rng.choice([0.0, 0.1]) if N > 64 else 0.0)
    K, m = _size(rng, 8, 65536), rng.choice([1, 2, 3, 4, 8])
    N = _log(rng, 1, min(1000003, MOST // (K * SIZE[dtype])))
    return dict(op=op, direction=rng.choice(["forward", "backward"]), N=N, K=K, m=m, dtype=dtype,
                normalised=m > 1 and rng.choice([False, True]),  # one weight that is always 1 has no gradient
                drop=rng.choice([0.0, 0.1]) if N > 64 else 0.0, masked=rng.choice([0.0, 0.2]))


# ----------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _logits(case, g):
    """A row's logits: components are unevenly popular, and a row prefers a few."""
    L = _randn(g, case["N"], case["K"]).mul_(1.5)
    return L.add_(_randn(g, case["K"]) * 0.5)


def _distinct(N, m, K, g):
    """m distinct ids of each row, the first of them anywhere."""
    first = torch.randint(0, K, (N, 1), device="cuda", generator=g)
    step = 1 + torch.randint(0, max(1, K // m), (N, m), device="cuda", generator=g)
    step[:, 0] = 0
    return (first + torch.cumsum(step, 1)) % K


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s, dt, N = {"case": dict(case), "own": {}}, DT[case["dtype"]], case["N"]
    if case["op"] == "norm":
        D, wt = case["D"], DT[case["weights"]]
        scale = torch.exp(0.3 * _randn(g, D))  # features differ in size, rows in mean
        s["X"] = (_randn(g, N, D).mul_(scale).add_(0.5 * _randn(g, N, 1))).to(dt)
        s["w"], s["b"] = (1 + 0.1 * _randn(g, D)).to(wt), (0.1 * _randn(g, D)).to(wt)
        if case["direction"] == "backward":
            s["dY"] = _randn(g, N, D).mul_(0.01).to(dt)
        return s
    K, m = case["K"], case["m"]
    L = _logits(case, g)
    if case["op"] == "distill":
        ids = _distinct(N, m, K, g)
        top = (6.0 + 2.0 * _randn(g, N, m)).sort(1, descending=True)[0]
        L.scatter_add_(1, ids, 0.7 * top + _randn(g, N, m))  # the student knows some of it
        s["logits"] = L.to(dt)
        s["ids"] = ids.to(torch.int32)
        s["values"] = top if case["teacher"] == "logits" else (torch.softmax(top, 1) * 0.98).contiguous()
        s["weights"] = None
        if case["drop"] > 0:  # entries that the teacher left out, and rows of padding
            s["ids"][:, 1:][torch.rand(N, m - 1, device="cuda", generator=g) < 0.1] = -1
            s["weights"] = torch.rand(N, device="cuda", generator=g) + 0.5
            s["weights"][torch.rand(N, device="cuda", generator=g) < case["drop"]] = 0.0
        return s
    if case["masked"] > 0:  # components that are not in use
        off = torch.rand(K, device="cuda", generator=g) < case["masked"]
        off[0] = False
        L.masked_fill_(off, float("-inf"))
    s["logits"], s["live"] = L.to(dt), None
    if case["drop"] > 0:  # rows of padding
        s["live"] = torch.rand(N, device="cuda", generator=g) >= case["drop"]
    if case["direction"] == "backward":
        s["ids"], s["gamma"], _, p = _gate(s)
        s["dgamma"] = _randn(g, N, m) * scale_of(case)
        s["share"] = None
        if case["op"] == "balance":
            counts, rows = _count(s["ids"], K), _rows(s)
            s["share"] = (K * counts.double() / (counts.sum() * rows).clamp(min=1)).float()
    return s


# -------------------------------------------------------------------- run

def _rows(s):
    """How many rows count."""
    some = torch.isfinite(s["logits"]).any(1)
    return (some if s["live"] is None else some & s["live"]).sum()


def _count(ids, K):
    flat = ids.reshape(-1).long()
    kept = (flat >= 0).long()
    return torch.zeros(K, dtype=torch.int64, device=ids.device).scatter_add_(0, flat.clamp(min=0), kept)


def _softmax(x):
    """Rows' exp(x - max) over their sum, and their log-sum-exp; a row of -inf has zeros."""
    top = x.amax(1, keepdim=True)
    low = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = torch.exp(x - low)
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, torch.ones_like(total)), (low + torch.log(total))[:, 0]


def _gate(s):
    """ids, gamma, lse and p."""
    c = s["case"]
    x = s["logits"].float()
    if s["live"] is not None:
        x = x.masked_fill(~s["live"][:, None], float("-inf"))
    value, ids = torch.sort(x, dim=1, descending=True, stable=True)
    value, ids = value[:, :c["m"]], ids[:, :c["m"]]
    p, lse = _softmax(x)
    if c["normalised"]:
        gamma = _softmax(value)[0]
    else:
        gamma = torch.gather(p, 1, ids)
    ids = torch.where(value > float("-inf"), ids, torch.full_like(ids, -1))
    return ids.to(torch.int32).contiguous(), gamma.contiguous(), lse, p


def _plain(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    if c["op"] == "norm":
        x = s["X"].float()
        x = x - x.mean(1, keepdim=True)
        rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        x = x * rstd
        if c["direction"] == "forward":
            return {"Y": (x * s["w"].float() + s["b"].float()).to(dt)}
        dy = s["dY"].float()
        dw, db = (dy * x).sum(0), dy.sum(0)
        g = dy * s["w"].float()
        dx = (g - g.mean(1, keepdim=True) - x * (g * x).mean(1, keepdim=True)) * rstd
        wt = s["w"].dtype
        return {"dX": dx.to(dt), "dw": dw.to(wt), "db": db.to(wt)}
    if c["op"] == "distill":
        T, N = c["T"], c["N"]
        p, lse = _softmax(s["logits"].float() / T)
        kept = s["ids"] >= 0
        at = s["ids"].long().clamp(min=0)
        t = (s["values"] if c["teacher"] == "logits" else torch.log(s["values"])) / T
        t = t.masked_fill(~kept, float("-inf"))
        q, total = _softmax(t)
        logq = (t - total[:, None]).masked_fill(~kept, 0.0)
        logp = torch.gather(s["logits"].float(), 1, at) / T - lse[:, None]
        rows = T * T * (q * (logq - logp)).sum(1)
        if s["weights"] is not None:
            rows = rows * s["weights"]
        out = {"rows": rows, "loss": rows.sum() * scale_of(c)}
        if c["direction"] == "step":
            d = p.scatter_add_(1, at, -q)
            w = torch.full((N, 1), T * scale_of(c), device=d.device)
            if s["weights"] is not None:
                w = w * s["weights"][:, None]
            out["dlogits"] = (d * w).to(dt)
        return out
    if c["direction"] == "forward":
        ids, gamma, lse, p = _gate(s)
        out = {"ids": ids, "gamma": gamma, "lse": lse}
        if c["op"] == "balance":
            counts, mass = _count(ids, c["K"]), p.sum(0)
            share = c["K"] * counts.float() / (counts.sum() * _rows(s)).clamp(min=1).float()
            out.update(counts=counts, mass=mass, loss=(share * mass).sum())
        return out
    x = s["logits"].float()
    if s["live"] is not None:
        x = x.masked_fill(~s["live"][:, None], float("-inf"))
    at = s["ids"].long().clamp(min=0)
    kept = s["ids"] >= 0
    v = s["dgamma"] * s["gamma"] * kept
    p = _softmax(x)[0]
    if c["normalised"]:
        v = v - s["gamma"] * kept * v.sum(1, keepdim=True)
        d = torch.zeros_like(p)
    else:
        d = -p * v.sum(1, keepdim=True)
    if c["op"] == "balance":
        share = coef_of(c) * s["share"]
        d += p * (share - (p * share).sum(1, keepdim=True))
    return {"dlogits": d.scatter_add_(1, at, v).to(dt)}


def _own(s):
    import soft_clustering_gb300 as G

    c, h = s["case"], s["own"]
    dt = DT[c["dtype"]]
    if c["op"] == "norm":
        from soft_clustering_gb300.norm import LayerNorm
        if not h:
            h["norm"] = LayerNorm(c["D"], dt, eps=EPS, weight_dtype=DT[c["weights"]])
        if c["direction"] == "forward":
            return {"Y": h["norm"].forward(s["X"], s["w"], s["b"])}
        dX, dw, db = h["norm"].backward(s["dY"], s["X"], s["w"])
        return {"dX": dX, "dw": dw, "db": db}
    from soft_clustering_gb300.gate import Distiller, Gate
    if c["op"] == "distill":
        if not h:
            h["distiller"] = Distiller(c["N"], c["K"], c["m"], dt, teacher=c["teacher"], temperature=c["T"], scale=scale_of(c))
        d = h["distiller"]
        if c["direction"] == "forward":
            return {"rows": d.rows, "loss": d.loss(s["logits"], s["ids"], s["values"], weights=s["weights"])[0]}
        loss, dlogits = d.step(s["logits"], s["ids"], s["values"], weights=s["weights"])
        return {"rows": d.rows, "loss": loss[0], "dlogits": dlogits}
    if c["direction"] == "forward":
        if not h:
            h["gate"] = Gate(c["N"], c["K"], c["m"], dt, normalised=c["normalised"])
        g = h["gate"]
        ids, gamma = g.forward(s["logits"], live=s["live"], balance=c["op"] == "balance")
        out = {"ids": ids, "gamma": gamma, "lse": g.lse}
        if c["op"] == "balance":
            out.update(counts=g.counts, mass=g.mass, loss=g.loss[0])
        return out
    dlogits = torch.empty_like(s["logits"])
    G.gmm_gate_grad(s["logits"], CODE[c["dtype"]], c["N"], c["K"], c["m"], int(c["normalised"]), s["live"], s["ids"], s["gamma"], s["dgamma"],
                    s["share"], coef_of(c) if c["op"] == "balance" else 0.0, dlogits)
    return {"dlogits": dlogits}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- work

def work(case):
    N, es = case["N"], SIZE[case["dtype"]]
    if case["op"] == "norm":
        D, wb = case["D"], SIZE[case["weights"]] * case["D"]
        if case["direction"] == "forward":
            return {"bytes": 2.0 * N * D * es + 2 * wb, "flops": 7.0 * N * D}
        return {"bytes": 3.0 * N * D * es + 3 * wb, "flops": 16.0 * N * D}
    K, m = case["K"], case["m"]
    live = N * (1 - case["drop"])  # rows that have to be read
    if case["op"] == "distill":
        teacher = 8.0 * N * m + 4 * N + (4 * N if case["drop"] else 0)
        if case["direction"] == "forward":
            return {"bytes": teacher + live * K * es + 4, "flops": 4.0 * live * K}
        return {"bytes": teacher + (live + N) * K * es + 4, "flops": 7.0 * live * K}
    small = 8.0 * N * m + (N if case["drop"] else 0)
    if case["direction"] == "forward":
        more = 12.0 * K + 4 if case["op"] == "balance" else 0.0
        return {"bytes": small + 4 * N + more + live * K * es, "flops": (5.0 + m) * live * K}
    more = 4.0 * K if case["op"] == "balance" else 0.0
    read = 0 if case["normalised"] and case["op"] == "gate" else live * K * es  # its gradient is of the kept entries alone
    return {"bytes": small + 4 * N * m + more + read + N * K * es, "flops": 6.0 * live * K}


# ------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        x, w = s["X"].to(f), s["w"].to(f)
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        h = (x - mean) / (var + EPS).sqrt()
        if case["direction"] == "forward":
            return {"Y": torch.addcmul(s["b"].to(f), h, w)}
        dy = s["dY"].to(f)
        dw, db = torch.einsum("nd,nd->d", dy, h), dy.sum(0)
        g = dy.mul_(w)
        along = torch.einsum("nd,nd->n", g, h)[:, None] / case["D"]
        dx = g.sub_(g.mean(1, keepdim=True)).addcmul_(h, along, value=-1.0).div_((var + EPS).sqrt())
        return {"dX": dx, "dw": dw, "db": db}
    x = s["logits"].to(f)
    if case["op"] == "distill":
        T, N = case["T"], case["N"]
        logp = torch.log_softmax(x / T, 1)
        v = s["values"].to(f)
        weight = (v / T).exp() if case["teacher"] == "logits" else v ** (1 / T)
        weight = torch.where(s["ids"] >= 0, weight, torch.zeros_like(weight))
        q = weight / weight.sum(1, keepdim=True)
        at = s["ids"].long().clamp(min=0)
        kl = (torch.xlogy(q, q) - q * logp.gather(1, at)).sum(1)
        w = torch.ones(N, dtype=f, device="cuda") if s["weights"] is None else s["weights"].to(f)
        rows = kl * w * T ** 2
        out = {"rows": rows, "loss": rows.sum() * scale_of(case)}
        if case["direction"] == "step":
            out["dlogits"] = logp.exp_().scatter_add_(1, at, -q).mul_(w[:, None] * (T * scale_of(case)))
        return out
    if s["live"] is not None:
        x[~s["live"]] = float("-inf")
    lse = torch.logsumexp(x, 1)
    none = torch.isneginf(lse)
    p = torch.exp(x - lse.masked_fill(none, 0.0)[:, None])
    if case["direction"] == "forward":
        gamma = torch.topk(p, case["m"], dim=1)[0]
        if case["normalised"]:
            gamma = gamma / gamma.sum(1, keepdim=True).masked_fill(none[:, None], 1.0)
        out = {"ids": None, "gamma": gamma, "lse": lse}
        if case["op"] == "balance":
            mass = p.sum(0)
            # counts of the m largest logits, ties to the lower component, as a plain form has them
            counts = torch.bincount(_gate(s)[0].reshape(-1).long() + 1, minlength=case["K"] + 1)[1:].to(f)
            loss = case["K"] * torch.dot(counts, mass) / (counts.sum() * (~none).sum()).clamp(min=1)
            out.update(counts=None, mass=mass, loss=loss)
        return out
    g = torch.zeros_like(p)
    at, kept = s["ids"].long().clamp(min=0), (s["ids"] >= 0).to(f)
    dg = s["dgamma"].to(f) * kept
    if case["normalised"]:
        # gamma_t = p_t / sum of the kept p: its own softmax
        own_p = p.gather(1, at) * kept
        own_p = own_p / own_p.sum(1, keepdim=True).masked_fill(none[:, None], 1.0)
        g.scatter_add_(1, at, own_p * (dg - torch.einsum("nm,nm->n", own_p, dg)[:, None]))
    else:
        full = torch.zeros_like(p).scatter_add_(1, at, dg)
        g = p * (full - torch.einsum("nk,nk->n", p, full)[:, None])
    if case["op"] == "balance":
        share = coef_of(case) * s["share"].to(f)
        g += p * (share - (p @ share)[:, None])
    return {"dlogits": g}
