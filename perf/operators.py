"""The score-matrix operators as they are measured: cases, inputs, one pass in plain torch or through the library, and
the same result in 64 bits.

Three operators on a given row-major score matrix: token log-probabilities (``scores_logprobs``, with
``scores_logprobs_grad``), routing to experts (``scores_route``, with ``scores_route_grad``) and the balancing Sinkhorn
potentials of a router's scores (``scores_solve``).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------------------------- cases

def _logprobs(name, n, m, dtype, top, entropy, train=False, eps=1.0, pad=0, masked=False):
    """pad: extra columns of the row stride; masked: most of each row is -inf (constrained decoding)."""
    return dict(name=name, op="logprobs", n=n, m=m, dtype=dtype, top=top, entropy=entropy, train=train, eps=eps, pad=pad,
                masked=masked)


def _route(name, n, m, dtype, k, fn, bias, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0, train=False, pad=0):
    """bias: "none", "score" (added to the activated score) or "logit" (added to the raw score)."""
    return dict(name=name, op="route", n=n, m=m, dtype=dtype, k=k, fn=fn, bias=bias, n_group=n_group, topk_group=topk_group,
                group_top=group_top, renorm=renorm, scale=scale, train=train, pad=pad)


def _solve(name, n, m, dtype, eps, iters, weighted=False, pad=0):
    """weighted: nonuniform expert capacities and padding tokens of weight zero."""
    return dict(name=name, op="solve", n=n, m=m, dtype=dtype, eps=eps, iters=iters, weighted=weighted, pad=pad)


def listed():
    return [
        # a single decoding step with the top alternatives that a serving interface returns
        _logprobs("logprobs_one_row", 1, 131072, "bf16", 20, True),
        # a decoding batch over an odd vocabulary, rows at odd offsets, sampling temperature
        _logprobs("logprobs_batch_odd", 64, 50001, "f32", 5, True, eps=0.7),
        # constrained decoding: a mask leaves about one token in five hundred
        _logprobs("logprobs_masked", 32, 65536, "f16", 20, False, masked=True),
        # scoring long prompts: given tokens only
        _logprobs("logprobs_prompt", 8192, 65536, "bf16", 0, False),
        # a policy-gradient step: log-probabilities, entropy bonus and their gradient
        _logprobs("logprobs_train", 4096, 65536, "bf16", 0, True, train=True),
        # a small head in 32 bits, odd sizes, gradient through the alternatives as in distillation
        _logprobs("logprobs_train_odd", 777, 2049, "f32", 8, True, train=True, pad=3),
        # one token of a small mixture
        _route("route_one_token", 1, 64, "f32", 6, "softmax", "none", renorm=False, scale=1.5),
        # a prompt through a large mixture: sigmoid scores, a bias for balance, groups
        _route("route_groups", 16384, 256, "f32", 8, "sigmoid", "score", 8, 4, 2, True, 2.5),
        # a training batch of a medium mixture with the gradient
        _route("route_train", 32768, 128, "bf16", 8, "softmax", "logit", renorm=False, train=True),
        # a batch of a small odd mixture with the gradient, padded rows
        _route("route_train_odd", 4099, 60, "f32", 4, "sigmoid", "score", renorm=True, train=True, pad=5),
        # balancing one decoding batch
        _solve("solve_small", 200, 16, "f32", 0.5, 8),
        # balancing a training batch of a large mixture, capacities and padding
        _solve("solve_batch", 32768, 256, "bf16", 0.25, 10, weighted=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "route", "solve"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    pad = rng.choice([0, 0, 1, 8, 13])
    if op == "logprobs":
        m = _log_int(rng, 32, 200000)
        train = rng.random() < 0.4
        n = _log_int(rng, 1, max(1, min(8192, (100_000_000 if train else 250_000_000) // m)))
        top = min(m, rng.choice([0, 1, 5, 20, 64]))
        if top and n * m > 20_000_000:
            n = max(1, 20_000_000 // m)
        c = _logprobs("", n, m, dtype, top, rng.random() < 0.5, train, rng.choice([1.0, 0.7, 1.3]), pad, rng.random() < 0.2)
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        m = groups * _log_int(rng, 4, 1024 // groups)
        topg = rng.randint(1, groups)
        k = rng.randint(1, min(16, topg * (m // groups)))
        n = _log_int(rng, 1, min(65536, 4_000_000 // m))
        fn, bias = rng.choice(["softmax", "sigmoid"]), rng.choice(["none", "score", "logit"])
        c = _route("", n, m, dtype, k, fn, bias, groups, topg, rng.choice([1, 2]), rng.random() < 0.6,
                   rng.choice([1.0, 2.5]), rng.random() < 0.5, pad)
    else:
        m = _log_int(rng, 4, 1024)
        n = _log_int(rng, 1, min(65536, 8_000_000 // m))
        c = _solve("", n, m, dtype, rng.choice([0.1, 0.25, 0.5, 1.0]), rng.randint(1, 12), rng.random() < 0.5, pad)
    del c["name"]
    return c


def work(case):
    n, m, es = case["n"], case["m"], SIZE[case["dtype"]]
    if case["op"] == "logprobs":
        out = n * (8 + 4 + 4 + (4 if case["entropy"] else 0) + 8 * case["top"])
        reads, writes = (2, 1) if case["train"] else (1, 0)
        return {"bytes": n * m * es * (reads + writes) + out, "flops": n * m * (14 if case["train"] else 6)}
    if case["op"] == "route":
        grads = n * m * es * (2 if case["fn"] == "softmax" and not case["renorm"] else 1) if case["train"] else 0
        return {"bytes": n * m * es + 8 * n * case["k"] + 4 * m + grads, "flops": n * m * (4 + case["k"])}
    # every iteration needs every score: the matrix is read once, and worked through once an iteration
    return {"bytes": n * m * es + 4 * (n + m) * (2 if case["weighted"] else 1), "flops": n * m * 6 * case["iters"]}


# ------------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    n, m, dtype = case["n"], case["m"], DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    st = dict(case=case)
    buf = torch.zeros((n, m + case["pad"]), dtype=dtype, device=dev)
    s = buf[:, :m]
    if case["op"] == "logprobs":
        tgt = torch.randint(0, m, (n,), generator=gen, device=dev)
        rows = torch.arange(n, device=dev)
        step = max(1, 50_000_000 // m)
        for r in range(0, n, step):  # a slab at a time: the random numbers are in 32 bits
            part = randn(min(step, n - r), m) * 2.5
            if case["masked"]:
                part.masked_fill_(rand(*part.shape) > 0.002 + 8.0 / m, -math.inf)
            s[r:r + step] = part.to(dtype)
        s[rows, tgt] = (6.0 + 3.0 * randn(n)).to(dtype)  # the given tokens are likely ones
        if n > 16:
            tgt[torch.randint(0, n, (n // 16,), generator=gen, device=dev)] = -1  # positions without a token
        st.update(scores=s, targets=tgt, d_logp=randn(n) / n)
        if case["train"]:
            if case["entropy"]:
                st["d_entropy"] = 0.01 * randn(n)
            if case["top"]:
                st["d_top"] = randn(n, case["top"]) / n
    elif case["op"] == "route":
        s.copy_((randn(n, m) + 0.5 * randn(1, m)).to(dtype))
        st.update(scores=s, bias=None if case["bias"] == "none" else 0.1 * randn(m))
        if case["train"]:
            st["d_weights"] = randn(n, case["k"])
    else:
        s.copy_((randn(n, m) + randn(1, m)).to(dtype))
        st.update(scores=s, a=None, b=None)
        if case["weighted"]:
            a = (rand(n) > 0.1).float()
            a[0] = 1.0
            b = 0.5 + rand(m)
            st.update(a=a / a.sum(), b=b / b.sum())
    return st


# ----------------------------------------------------------------------------------------- the plain form, 32 bits

def _lse(z, dim):
    """log-sum-exp with the maximum taken out; -inf where nothing is left."""
    top = z.amax(dim, keepdim=True).clamp_min(-3.0e38)
    return (top + (z - top).exp().sum(dim, keepdim=True).log()).squeeze(dim)


def _top(v, k):
    """The k largest of each row in descending order, ties to the lowest index."""
    bits = (v + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    place = 0xFFFFFFFF - torch.arange(v.shape[1], device=v.device)
    return (0xFFFFFFFF - ((order << 32) | place).topk(k, dim=1).values.bitwise_and(0xFFFFFFFF)).long()


def _plain_logprobs(st):
    c, s, tgt, eps = st["case"], st["scores"].float(), st["targets"], st["case"]["eps"]
    given = tgt >= 0
    at = tgt.clamp_min(0)[:, None]
    top = s.amax(1, keepdim=True).clamp_min(-3.0e38)
    d = (s - top) / eps
    e = d.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    out = {"logp": torch.where(given, (d.gather(1, at) - log_total)[:, 0], torch.zeros(())),
           "lse": (top / eps + log_total)[:, 0]}
    if c["entropy"]:
        mean_d = (e * torch.where(e > 0, d, torch.zeros(()))).sum(1, keepdim=True) / total
        out["entropy"] = (log_total - mean_d)[:, 0]
    if c["top"]:
        idx = _top(s, c["top"])
        out["top_idx"], out["top_logp"] = idx.int(), d.gather(1, idx) - log_total
    if c["train"]:
        p = e / total
        g = torch.where(given, st["d_logp"], torch.zeros(()))[:, None]
        pull = g.clone()
        if c["top"]:
            pull = pull + st["d_top"].sum(1, keepdim=True)
        dz = -p * pull
        if c["entropy"]:
            dz -= torch.where(p > 0, p * (d - mean_d), torch.zeros(())) * st["d_entropy"][:, None]
        dz.scatter_add_(1, at, g)
        if c["top"]:
            dz.scatter_add_(1, idx, st["d_top"])
        out["grad"] = (dz / eps).to(st["scores"].dtype)
    return out


def _choice(st):
    """The experts chosen for each token; their values lie next to each other, so these are taken in 64 bits."""
    c, s, (n, m) = st["case"], st["scores"].double(), st["scores"].shape
    v = s
    if c["bias"] == "score" or (c["bias"] == "none" and c["group_top"] == 2):
        v = torch.sigmoid(s) if c["fn"] == "sigmoid" else torch.softmax(s, 1)
    if st["bias"] is not None:
        v = v + st["bias"].double()
    if c["n_group"] > 1:
        per = v.view(n, c["n_group"], m // c["n_group"])
        score = per.sort(2, descending=True).values[:, :, :c["group_top"]].sum(2)
        best = score.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        v = torch.where(keep[:, :, None], per, -math.inf).reshape(n, m)
    return v.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]


def _plain_route(st):
    c, s, m = st["case"], st["scores"].float(), st["scores"].shape[1]
    idx = _choice(st)
    picked = s.gather(1, idx)
    if c["fn"] == "sigmoid":
        log_act = -torch.log1p((-picked.abs()).exp()) + picked.clamp_max(0.0)
    else:
        log_act = picked - _lse(s, 1)[:, None]
    if c["renorm"]:
        log_act = log_act - _lse(log_act, 1)[:, None]
    q = log_act.exp()
    out = {"idx": idx.int(), "weights": q * c["scale"],
           "counts": torch.zeros(m, dtype=torch.int32, device=s.device).scatter_add_(
               0, idx.reshape(-1), torch.ones((), dtype=torch.int32, device=s.device).expand(idx.numel()))}
    if c["train"]:
        dq = st["d_weights"] * c["scale"]
        inner = (q * dq).sum(1, keepdim=True)
        if c["fn"] == "sigmoid":
            rest = torch.sigmoid(-picked)
            ds = torch.zeros_like(s).scatter_(1, idx, q * ((dq - inner) if c["renorm"] else dq) * rest)
        elif c["renorm"]:
            ds = torch.zeros_like(s).scatter_(1, idx, q * (dq - inner))
        else:
            ds = -(s - _lse(s, 1)[:, None]).exp() * inner
            ds.scatter_add_(1, idx, q * dq)
        out["grad"] = ds.to(st["scores"].dtype)
    return out


def _plain_solve(st):
    c, s, (n, m) = st["case"], st["scores"].float(), st["scores"].shape
    eps = c["eps"]
    log_a = torch.full((n,), -math.log(n), device=s.device) if st["a"] is None else st["a"].log()
    log_b = torch.full((m,), -math.log(m), device=s.device) if st["b"] is None else st["b"].log()
    f, g = torch.zeros(n, device=s.device), torch.zeros(m, device=s.device)
    for _ in range(c["iters"]):
        f = -eps * _lse((g + s) / eps + log_b, 1)
        g = -eps * _lse((f[:, None] + s) / eps + log_a[:, None], 0)
    return {"f": f, "g": g}


# --------------------------------------------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if not own:
        return {"logprobs": _plain_logprobs, "route": _plain_route, "solve": _plain_solve}[c["op"]](st)
    import streaming_sinkhorn_solver_amd as sk

    s = st["scores"]
    if c["op"] == "logprobs":
        r = sk.scores_logprobs(s, st["targets"], eps=c["eps"], top=c["top"], entropy=c["entropy"])
        out = {"logp": r.logp, "lse": r.lse}
        if c["entropy"]:
            out["entropy"] = r.entropy
        if c["top"]:
            out["top_idx"], out["top_logp"] = r.top_idx, r.top_logp
        if c["train"]:
            out["grad"] = sk.scores_logprobs_grad(s, st["targets"], r, eps=c["eps"], d_logp=st["d_logp"],
                                                  d_entropy=st.get("d_entropy"), d_top=st.get("d_top"))
        return out
    if c["op"] == "route":
        how = dict(score_fn=c["fn"], renorm=c["renorm"], scale=c["scale"])
        r = sk.scores_route(s, c["k"], bias=st["bias"], select_on="logit" if c["bias"] == "logit" else "score",
                            n_group=c["n_group"], topk_group=c["topk_group"], group_top=c["group_top"], counts=True, **how)
        out = {"idx": r.idx, "weights": r.weights, "counts": r.counts}
        if c["train"]:
            out["grad"] = sk.scores_route_grad(s, r.idx, st["d_weights"], **how)
        return out
    f, g = sk.scores_solve(s, st["a"], st["b"], eps=c["eps"], n_iters=c["iters"], check=False)
    return {"f": f, "g": g}


# ------------------------------------------------------------------------------- the same from the definition, 64 bits

def _exact_logprobs(case, st):
    eps, top_k = case["eps"], case["top"]
    out = {k: [] for k in ("logp", "lse", "entropy", "top_idx", "top_logp", "grad")}
    step = max(1, 20_000_000 // case["m"])
    for r in range(0, case["n"], step):
        z = st["scores"][r:r + step].double() / eps
        t = st["targets"][r:r + step]
        logp = torch.log_softmax(z, 1)
        p = logp.exp()
        plogp = torch.special.xlogy(p, p)
        hot = torch.zeros_like(z)
        hot[t >= 0, t[t >= 0]] = 1.0
        out["logp"].append(torch.where(t >= 0, logp.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0))
        out["lse"].append(torch.logsumexp(z, 1))
        h = -plogp.sum(1)
        out["entropy"].append(h)
        if top_k:
            value, idx = torch.sort(st["scores"][r:r + step].double(), dim=1, descending=True, stable=True)
            idx = idx[:, :top_k]
            out["top_idx"].append(idx.int())
            out["top_logp"].append(logp.gather(1, idx))
        if case["train"]:
            dz = (hot - p * (t >= 0)[:, None]) * st["d_logp"][r:r + step].double()[:, None]
            if case["entropy"]:
                dz -= (plogp + p * h[:, None]) * st["d_entropy"][r:r + step].double()[:, None]
            if top_k:
                dt = st["d_top"][r:r + step].double()
                dz.scatter_add_(1, idx, dt)
                dz -= p * dt.sum(1, keepdim=True)
            out["grad"].append(dz / eps)
    keep = ["logp", "lse"] + ["entropy"] * case["entropy"] + ["top_idx", "top_logp"] * bool(top_k) + ["grad"] * case["train"]
    return {k: torch.cat(out[k]) for k in keep}


def _exact_route(case, st):
    s = st["scores"].double().requires_grad_(case["train"])
    act = torch.sigmoid(s) if case["fn"] == "sigmoid" else torch.softmax(s, 1)
    with torch.no_grad():
        raw = case["bias"] == "logit" or (case["bias"] == "none" and case["group_top"] == 1)
        v = s.detach() if raw else act.detach()
        v = v + (0.0 if st["bias"] is None else st["bias"].double())
        size = case["m"] // case["n_group"]
        if case["n_group"] > 1:
            score = torch.stack([torch.topk(b, min(case["group_top"], size), 1).values.sum(1) for b in v.split(size, 1)], 1)
            order = torch.sort(-score, dim=1, stable=True).indices
            v = v.clone()
            for lost in range(case["topk_group"], case["n_group"]):
                cols = order[:, lost:lost + 1] * size + torch.arange(size, device=v.device)
                v.scatter_(1, cols, -math.inf)
        idx = torch.sort(-v, dim=1, stable=True).indices[:, :case["k"]]
    w = act.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    out = {"idx": idx.int(), "weights": w.detach(),
           "counts": torch.bincount(idx.reshape(-1), minlength=case["m"]).int()}
    if case["train"]:
        out["grad"] = torch.autograd.grad(w, s, st["d_weights"].double())[0]
    return out


def _exact_solve(case, st):
    n, m, eps = case["n"], case["m"], case["eps"]
    z = st["scores"].double() / eps
    log_a = torch.log(torch.full((n,), 1.0 / n, device=z.device).double() if st["a"] is None else st["a"].double())
    log_b = torch.log(torch.full((m,), 1.0 / m, device=z.device).double() if st["b"] is None else st["b"].double())
    u, v = torch.zeros(n, device=z.device).double(), torch.zeros(m, device=z.device).double()
    for _ in range(case["iters"]):
        u = -torch.logsumexp(z + (v + log_b)[None, :], 1)
        v = -torch.logsumexp(z + (u + log_a)[:, None], 0)
    return {"f": eps * u, "g": eps * v}


def exact(case, seed):
    st = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "route": _exact_route, "solve": _exact_solve}[case["op"]](case, st)
