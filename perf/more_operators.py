"""Operators behind the router and the head as they are measured: cases, inputs, one pass in plain torch or through the
library, and the same result in 64 bits.

Token rows sorted by expert and back (``route_sort``, ``route_dispatch``, ``route_combine``, ``route_combine_grad``), and
the verification of drafted tokens from given random numbers (``scores_verify``).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------------------------- cases

def _route(name, op, n, k, m, d=0, dtype="bf16", align=1, capacity=0, dropped=0.0, weighted=False, add=False, pad=0):
    """op: "sort" (the plan alone), "dispatch" (the plan and the sorted rows), "combine" (back, weighted) or "grad" (the
    gradients of the last two).  capacity: rows that an expert takes at most (0: any); dropped: share of the choices
    that lie with experts of other devices; weighted: weights on the way out; add: a shared expert's output is added;
    pad: extra columns of the tokens' row stride."""
    return dict(name=name, op=op, n=n, k=k, m=m, d=d, dtype=dtype, align=align, capacity=capacity, dropped=dropped,
                weighted=weighted, add=add, pad=pad)


def _verify(name, b, drafts, m, dtype, draft, eps=1.0, eps_draft=1.0, ragged=False, padded=False, masked=False, pad=0):
    """b requests of up to `drafts` drafted tokens and one row more; draft: the draft model's scores are given; eps 0:
    greedy; ragged: requests of different lengths, packed, or (padded) each in drafts + 1 rows; masked: most of the
    vocabulary is ruled out; pad: extra columns of the row stride."""
    return dict(name=name, op="verify", b=b, drafts=drafts, m=m, dtype=dtype, draft=draft, eps=eps, eps_draft=eps_draft,
                ragged=ragged, padded=padded, masked=masked, pad=pad)


def listed():
    return [
        # a prompt's choices among many experts
        _route("sort_prompt", "sort", 16384, 8, 256),
        # a training batch on one of several devices: most choices lie elsewhere, tiles of 16 rows, limited capacity
        _route("sort_device", "sort", 50021, 6, 60, align=16, capacity=2048, dropped=0.7),
        # one token of a decoding step
        _route("dispatch_one_token", "dispatch", 1, 8, 64, 2048),
        # a prompt, segments in whole tiles
        _route("dispatch_prompt", "dispatch", 16384, 8, 256, 2048, align=16),
        # a decoding batch, with the shared expert's output
        _route("combine_step", "combine", 64, 8, 64, 2048, add=True),
        # a prompt in half precision
        _route("combine_prompt", "combine", 16384, 8, 128, 2048, "f16", add=True),
        # the backward pass of a training batch
        _route("grad_train", "grad", 16384, 8, 128, 2048),
        # a small odd layer in 32 bits, choices dropped by capacity, padded rows
        _route("grad_train_odd", "grad", 777, 3, 10, 1027, "f32", align=4, capacity=200, dropped=0.1, pad=3),
        # one request with four drafted tokens: the latency of a decoding step
        _verify("verify_one", 1, 4, 131072, "bf16", True),
        # a decoding batch, requests of different numbers of drafts
        _verify("verify_batch", 64, 7, 131072, "bf16", True, eps=0.8, ragged=True),
        # drafts looked up in the prompt (no draft scores), an odd vocabulary in 32 bits under a mask
        _verify("verify_lookup_odd", 24, 5, 50001, "f32", False, eps=0.7, ragged=True, padded=True, masked=True, pad=7),
        # greedy decoding
        _verify("verify_greedy", 128, 3, 65536, "f16", False, eps=0.0, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "grad", "verify", "verify"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    pad = rng.choice([0, 0, 1, 8, 13])
    if op == "verify":
        m = _log_int(rng, 32, 200000)
        drafts = rng.randint(0, 12)
        b = _log_int(rng, 1, max(1, min(512, 40_000_000 // (m * (drafts + 1)))))
        greedy = rng.random() < 0.2
        ragged = rng.random() < 0.6
        c = _verify("", b, drafts, m, dtype, not greedy and rng.random() < 0.7, 0.0 if greedy else rng.choice([1.0, 0.7, 1.3]),
                    rng.choice([1.0, 0.6]), ragged, ragged and rng.random() < 0.5, rng.random() < 0.2, pad)
    else:
        m = _log_int(rng, 2, 1024)
        k = rng.randint(1, min(m, 12))
        d = 0 if op == "sort" else _log_int(rng, 24, 8192)
        most = 400_000 if op == "sort" else 200_000_000 // (d * SIZE[dtype])
        n = _log_int(rng, 1, max(1, min(65536, most // k)))
        capacity = rng.choice([0, 0, 1 + 2 * n * k // m])
        c = _route("", op, n, k, m, d, dtype, rng.choice([1, 1, 8, 16, 64]), capacity, rng.choice([0.0, 0.0, 0.1, 0.6]),
                   op == "dispatch" and rng.random() < 0.3, op == "combine" and rng.random() < 0.5, pad)
    del c["name"]
    return c


def work(case):
    es = SIZE[case["dtype"]]
    if case["op"] == "verify":
        b, m = case["b"], case["m"]
        n = b * (case["drafts"] + 1) if not case["ragged"] else b * (case["drafts"] + 2) // 2  # (half of them in the mean)
        scores = n * m + ((n - b) * m if case["draft"] else 0)
        return {"bytes": scores * es + 28 * n + 24 * b, "flops": scores * (20 if case["eps"] else 1)}
    n, k, m, d = case["n"], case["k"], case["m"], case["d"]
    pairs = n * k
    plan = 12 * pairs + 8 * m
    if case["op"] == "sort":
        return {"bytes": plan, "flops": 2 * pairs}
    kept = pairs * (1.0 - case["dropped"])
    if case["capacity"]:
        kept = min(kept, m * case["capacity"])
    rows, tokens = int(kept * d), n * d
    if case["op"] == "dispatch":
        return {"bytes": (rows + tokens) * es + plan, "flops": rows if case["weighted"] else 0}
    if case["op"] == "combine":
        return {"bytes": (rows + tokens * (2 if case["add"] else 1)) * es + 8 * pairs, "flops": 2 * rows}
    # combine's gradient reads the rows and d_out, writes d_rows and d_weights; dispatch's reads rows and writes d_x
    return {"bytes": (3 * rows + 2 * tokens) * es + 12 * pairs, "flops": 4 * rows}


# ------------------------------------------------------------------------------------------------------ inputs

def _most_rows(case):
    """Rows that the sorted tokens can take: every segment is rounded up."""
    pairs, m, align, cap = case["n"] * case["k"], case["m"], case["align"], case["capacity"]
    rows = pairs + min(pairs, m) * (align - 1)
    return min(rows, m * ((cap + align - 1) // align * align)) if cap else rows


def _plain_sort(idx, case):
    """(slot, source, counts, offsets) by a stable sort."""
    n, k, m, align, cap = (case[c] for c in ("n", "k", "m", "align", "capacity"))
    e = idx.reshape(-1).long()
    e = torch.where((e >= 0) & (e < m), e, m)
    order = torch.sort(e, stable=True).indices
    sorted_e = e[order]
    seen = torch.zeros(m + 1, dtype=torch.long, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    first = seen.cumsum(0) - seen
    rank = torch.arange(n * k, device=e.device) - first[sorted_e]
    kept = sorted_e < m
    counts = seen[:m]
    if cap:
        kept &= rank < cap
        counts = counts.clamp_max(cap)
    ends = ((counts + align - 1) // align * align).cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    at = torch.where(kept, offsets[sorted_e] + rank, -1)
    slot = torch.empty_like(at).scatter_(0, order, at)
    rows = _most_rows(case)
    source = torch.full((rows + 1,), -1, dtype=torch.long, device=e.device)
    source.scatter_(0, torch.where(kept, at, rows), torch.where(kept, order, -1))
    return slot.view(n, k).int(), source[:rows].int(), counts.int(), offsets.int()


def _window(rows, cols, pad, dtype, dev):
    """A (rows, cols) window of a buffer whose rows are pad longer."""
    return torch.zeros((rows, cols + pad), dtype=dtype, device=dev)[:, :cols]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    st = dict(case=case)
    if case["op"] != "verify":
        n, k, m, d = (case[c] for c in ("n", "k", "m", "d"))
        # the choices of a router whose experts are not equally liked
        liked = (randn(n, m) + 0.7 * randn(1, m)).topk(k, dim=1)
        idx = liked.indices.int()
        if case["dropped"]:
            idx = torch.where(rand(n, k) < case["dropped"], torch.where(rand(n, k) < 0.5, -1, m), idx).int()
        st.update(idx=idx, weights=torch.softmax(liked.values, 1))
        if case["op"] == "sort":
            return st
        rows = _most_rows(case)
        x = _window(n, d, case["pad"], dtype, dev)
        x.copy_(randn(n, d))
        if case["op"] == "dispatch":
            # the rows behind the last segment are left as they are: the program's buffer starts as zeros
            st.update(x=x, rows=torch.zeros((rows, d), dtype=dtype, device=dev))
            return st
        expert_rows = torch.empty((rows, d), dtype=dtype, device=dev)
        step = max(1, 50_000_000 // max(d, 1))
        for r in range(0, rows, step):  # a slab at a time: the random numbers are in 32 bits
            expert_rows[r:r + step] = randn(min(step, rows - r), d).to(dtype)
        st.update(plan=_plain_sort(idx, case), rows=expert_rows)
        if case["op"] == "combine":
            st.update(add=x if case["add"] else None)
        else:
            st.update(d_y=x, d_rows=torch.zeros((rows, d), dtype=dtype, device=dev))
        return st

    b, m, most = case["b"], case["m"], case["drafts"]
    lengths = torch.full((b,), most, device=dev)  # drafted tokens of each request
    if case["ragged"]:
        lengths = torch.randint(0, most + 1, (b,), generator=gen, device=dev)
        if not case["padded"] and b > 1:  # about half of the rows, as work() counts them
            lengths[1::2] = most - lengths[:b // 2 * 2:2]
    taken = torch.full((b,), most + 1, device=dev) if case["padded"] else lengths + 1
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), taken.cumsum(0)])
    n = int(starts[-1])
    request = torch.repeat_interleave(torch.arange(b, device=dev), taken)
    place = torch.arange(n, device=dev) - starts[request]
    drafted = place < lengths[request]
    target = _window(n, m, case["pad"], dtype, dev)
    draft = _window(n, m, case["pad"], dtype, dev) if case["draft"] else None
    tokens = torch.full((n,), -1, dtype=torch.long, device=dev)
    step = max(1, 50_000_000 // m)
    for r in range(0, n, step):
        here = slice(r, min(n, r + step))
        size = here.stop - r
        logits = 2.0 * randn(size, m)
        if case["masked"]:
            ruled_out = rand(size, m) > 0.01 + 4.0 / m
            ruled_out[torch.arange(size, device=dev), torch.randint(0, m, (size,), generator=gen, device=dev)] = False
            logits = logits.masked_fill(ruled_out, -math.inf)
        near = logits + 0.5 * randn(size, m)  # the draft model is near the target model
        target[here] = logits.to(dtype)
        if draft is not None:
            draft[here] = near.to(dtype)
            likely = draft[here].float() / case["eps_draft"]
        else:
            likely = near
        noise = -torch.log(-torch.log(rand(size, m).clamp(1e-30, 1.0 - 1e-7)))
        tokens[here] = (likely + (0.1 if draft is None else 1.0) * noise).argmax(1)  # drawn from the draft's distribution
    tokens = torch.where(drafted, tokens, -1)
    st.update(target=target, draft=draft, tokens=tokens, starts=starts, u_accept=rand(n), u_sample=rand(b))
    return st


# ----------------------------------------------------------------------------------------- the plain form, 32 bits

def _plain_dispatch(x, slot, offsets, out, weights):
    n, k = slot.shape
    taken = torch.arange(out.shape[0], device=x.device) < offsets[-1]
    out = torch.where(taken[:, None], torch.zeros((), dtype=out.dtype, device=x.device), out)
    values = x.float()[:, None, :].expand(n, k, x.shape[1])
    if weights is not None:
        values = values * weights[:, :, None]
    kept = slot.reshape(-1) >= 0
    out[slot.reshape(-1)[kept].long()] = values.reshape(n * k, -1)[kept].to(out.dtype)
    return out


def _plain_combine(rows, slot, weights, add):
    y = torch.zeros((slot.shape[0], rows.shape[1]), device=rows.device) if add is None else add.float()
    for r in range(slot.shape[1]):
        kept = (slot[:, r] >= 0)[:, None]
        value = rows[slot[:, r].clamp_min(0).long()].float()
        if weights is not None:
            value = value * weights[:, r:r + 1]
        y = y + torch.where(kept, value, torch.zeros((), device=rows.device))
    return y.to(rows.dtype)


def _plain_combine_grad(rows, slot, offsets, weights, d_y, d_rows):
    d_weights = torch.empty_like(weights)
    for r in range(slot.shape[1]):
        value = rows[slot[:, r].clamp_min(0).long()].float()
        d_weights[:, r] = torch.where(slot[:, r] >= 0, (value * d_y.float()).sum(1), torch.zeros((), device=rows.device))
    return _plain_dispatch(d_y, slot, offsets, d_rows, weights), d_weights


def _plain_verify(st):
    """Accept / reject and the choice of a token lie next to borders: probabilities and their sums in 64 bits."""
    c, s, tok, starts = st["case"], st["target"].double(), st["tokens"], st["starts"]
    b = c["b"]
    n, m = s.shape
    dev = s.device
    rows = torch.arange(n, device=dev)
    top = s.amax(1, keepdim=True)
    if c["eps"] == 0.0:
        best = torch.where(s == top, torch.arange(m, device=dev), m).amin(1)
        p = torch.zeros_like(s)
        p[rows, best] = 1.0
    else:
        p = ((s - top) / c["eps"]).exp()
        p = p / p.sum(1, keepdim=True)
    at = tok.clamp_min(0)
    drafted = tok >= 0
    if st["draft"] is not None:
        t = st["draft"].double()
        q = ((t - t.amax(1, keepdim=True)) / c["eps_draft"]).exp()
        q = q / q.sum(1, keepdim=True)
        q = torch.where(drafted[:, None], q, 0.0)
    else:
        q = torch.zeros_like(s)
        q[rows[drafted], tok[drafted]] = 1.0
    taken = drafted & (st["u_accept"].double() * q[rows, at] < p[rows, at])
    # the first row of each request that is not taken
    refused = torch.where(taken, n, rows)
    request = torch.searchsorted(starts, rows, right=True) - 1
    stop = torch.full((b,), n, dtype=torch.long, device=dev).scatter_reduce(0, request, refused, "amin")
    found = stop < starts[1:]
    stop = torch.where(found, stop, starts[1:])
    accepted = stop - starts[:-1]
    row = stop.clamp_max(n - 1)
    r = (p[row] - q[row]).clamp_min(0.0)
    r = torch.where((r.sum(1) > 0.0)[:, None], r, p[row])
    total = r.cumsum(1)
    token = (total <= st["u_sample"].double()[:, None] * total[:, -1:]).sum(1)
    last = torch.where(r > 0.0, torch.arange(m, device=dev), -1).amax(1)  # (rounding: not behind the last possible one)
    token = torch.where(found, torch.minimum(token, last), -1)
    place = rows - starts[request]
    emitted = torch.where(place < accepted[request], tok, torch.where(place == accepted[request], token[request], -1))
    ratio = torch.where(drafted, (p[rows, at] / q[rows, at]).clamp_max(1.0), 0.0)
    logp = torch.where(emitted >= 0, p[rows, emitted.clamp_min(0)].log(), 0.0)
    return {"accepted": accepted.int(), "next": token, "tokens": emitted, "ratio": ratio.float(), "logp": logp.float()}


# --------------------------------------------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "verify":
            return _plain_verify(st)
        if op == "sort":
            return dict(zip(("slot", "source", "counts", "offsets"), _plain_sort(st["idx"], c)))
        if op == "dispatch":
            slot, source, counts, offsets = _plain_sort(st["idx"], c)
            rows = _plain_dispatch(st["x"], slot, offsets, st["rows"], st["weights"] if c["weighted"] else None)
            return {"slot": slot, "source": source, "counts": counts, "offsets": offsets, "rows": rows}
        slot, source, counts, offsets = st["plan"]
        if op == "combine":
            return {"y": _plain_combine(st["rows"], slot, st["weights"], st["add"])}
        d_rows, d_weights = _plain_combine_grad(st["rows"], slot, offsets, st["weights"], st["d_y"], st["d_rows"])
        # (the experts' own gradient lies between; here the rows' gradient goes back as it is)
        return {"d_rows": d_rows, "d_weights": d_weights, "d_x": _plain_combine(d_rows, slot, None, None)}
    import streaming_sinkhorn_solver_amd as sk

    if op == "verify":
        v = sk.scores_verify(st["target"], st["tokens"], st["starts"], st["u_accept"], st["u_sample"], draft=st["draft"],
                             eps=c["eps"], eps_draft=c["eps_draft"])
        return {"accepted": v.accepted, "next": v.next, "tokens": v.tokens, "ratio": v.ratio, "logp": v.logp}
    if op in ("sort", "dispatch"):
        plan = sk.route_sort(st["idx"], c["m"], align=c["align"], capacity=c["capacity"])
        out = {"slot": plan.slot, "source": plan.source, "counts": plan.counts, "offsets": plan.offsets}
        if op == "dispatch":
            out["rows"] = sk.route_dispatch(st["x"], plan, st["weights"] if c["weighted"] else None, out=st["rows"])
        return out
    plan = sk.RoutePlan(*st["plan"], align=c["align"])
    if op == "combine":
        return {"y": sk.route_combine(st["rows"], plan, st["weights"], add=st["add"])}
    d_rows, d_weights = sk.route_combine_grad(st["rows"], plan, st["weights"], st["d_y"], d_rows=st["d_rows"])
    return {"d_rows": d_rows, "d_weights": d_weights, "d_x": sk.route_combine(d_rows, plan)}


# ------------------------------------------------------------------------------- the same from the definition, 64 bits

def _exact_plan(idx, case):
    """Each expert's pairs in order, by comparison (no sort)."""
    n, k, m, align, cap = (case[c] for c in ("n", "k", "m", "align", "capacity"))
    flat = idx.flatten()
    slot = torch.full_like(flat, -1)
    source = torch.full((_most_rows(case),), -1, dtype=torch.int32, device=idx.device)
    counts, offsets, start = [], [0], 0
    for e in range(m):
        mine = (flat == e).nonzero()[:, 0]
        mine = mine[:cap] if cap else mine
        size = mine.numel()
        places = torch.arange(start, start + size, device=idx.device, dtype=torch.int32)
        slot[mine] = places
        source[start:start + size] = mine.int()
        start += -(-size // align) * align
        counts.append(size)
        offsets.append(start)
    return (slot.view(n, k), source, torch.tensor(counts, dtype=torch.int32, device=idx.device),
            torch.tensor(offsets, dtype=torch.int32, device=idx.device))


def _exact_rows(source, offsets, k, tokens, weights, behind):
    """Row by row from its pair: the token's row, weighted; zero where a segment is padded; what was there behind."""
    out = behind.double()
    end = int(offsets[-1])
    pair = source[:end].long()
    value = tokens.double().index_select(0, pair.clamp_min(0) // k)
    if weights is not None:
        value = value * weights.double().flatten()[pair.clamp_min(0)][:, None]
    out[:end] = value.masked_fill((pair < 0)[:, None], 0.0)
    return out


def _exact_back(source, n, k, rows, weights, add):
    """Each row added onto its token."""
    y = torch.zeros((n, rows.shape[1]), dtype=torch.float64, device=rows.device) if add is None else add.double()
    at = (source >= 0).nonzero()[:, 0]
    pair = source[at].long()
    step = max(1, 100_000_000 // max(rows.shape[1], 1))
    for r in range(0, at.numel(), step):
        value = rows[at[r:r + step]].double()
        if weights is not None:
            value *= weights.double().flatten()[pair[r:r + step]][:, None]
        y.index_add_(0, pair[r:r + step] // k, value)
    return y


def _exact_route(case, st):
    n, k = case["n"], case["k"]
    slot, source, counts, offsets = _exact_plan(st["idx"], case)
    out = {"slot": slot, "source": source, "counts": counts, "offsets": offsets}
    if case["op"] == "sort":
        return out
    if case["op"] == "dispatch":
        out["rows"] = _exact_rows(source, offsets, k, st["x"], st["weights"] if case["weighted"] else None, st["rows"])
        return out
    if case["op"] == "combine":
        return {"y": _exact_back(source, n, k, st["rows"], st["weights"], st["add"])}
    d_rows = _exact_rows(source, offsets, k, st["d_y"], st["weights"], st["d_rows"])
    d_weights = torch.zeros(n * k, dtype=torch.float64, device=slot.device)
    pairs = (slot.flatten() >= 0).nonzero()[:, 0]
    for part in pairs.split(max(1, 50_000_000 // case["d"])):
        rows = st["rows"][slot.flatten()[part].long()].double()
        d_weights[part] = torch.linalg.vecdot(rows, st["d_y"][part // k].double())
    # what goes back are the rows' gradients as they are held, in their type
    held = d_rows.to(st["rows"].dtype)
    return {"d_rows": d_rows, "d_weights": d_weights.view(n, k), "d_x": _exact_back(source, n, k, held, None, None)}


def _exact_verify(case, st):
    b, m = case["b"], case["m"]
    starts = st["starts"].tolist()
    tokens, u = st["tokens"].tolist(), st["u_accept"].double().tolist()
    dev = st["tokens"].device
    emitted = torch.full_like(st["tokens"], -1)
    ratio, logp = (torch.zeros(len(tokens), dtype=torch.float64, device=dev) for _ in range(2))
    accepted, after = [], []

    def log_p(scores, eps):
        if eps == 0.0:
            z = torch.full((m,), -math.inf, dtype=torch.float64, device=dev)
            z[(scores == scores.max()).nonzero()[0]] = 0.0
            return z
        z = scores.double() / eps
        return z - torch.logsumexp(z, 0)

    for r in range(b):
        count, token = 0, None
        for i in range(starts[r], starts[r + 1]):
            t = tokens[i]
            if t < 0 and token is not None:
                break
            lp = log_p(st["target"][i], case["eps"])
            rest = lp.exp()
            if t >= 0:
                if st["draft"] is None:
                    lq = torch.full_like(lp, -math.inf)
                    lq[t] = 0.0
                else:
                    lq = log_p(st["draft"][i], case["eps_draft"])
                odds = lp[t] - lq[t]
                ratio[i] = odds.clamp_max(0.0).exp()
                if token is not None:
                    continue
                if u[i] * math.exp(float(lq[t])) < math.exp(float(lp[t])):
                    emitted[i], logp[i] = t, lp[t]
                    count += 1
                    continue
                rest = torch.relu(rest - lq.exp())
                if not bool((rest > 0).any()):
                    rest = lp.exp()
            if token is None:
                mass = torch.cumsum(rest, 0)
                token = int(torch.searchsorted(mass, st["u_sample"][r:r + 1].double() * mass[-1], right=True).clamp_max(m - 1))
                emitted[i], logp[i] = token, lp[token]
        accepted.append(count)
        after.append(-1 if token is None else token)
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device=dev), "next": torch.tensor(after, device=dev),
            "tokens": emitted, "ratio": ratio, "logp": logp}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_verify(case, st) if case["op"] == "verify" else _exact_route(case, st)
