"""Measured cases of the layer norm, token log-probability and distillation operators.

Each operator is given twice: in a plain form of elementary torch operations in fp32
(``own`` false) and as the calls a user makes of this package (``own`` true), both on the
inputs that ``prepare`` builds; ``exact`` states the definition in float64.

Shapes: the norm runs on this library's own gate inputs ([220000, 512], [16384, 4096] and
odd ones), the vocabulary operators on generic vocabularies from a few hundred entries to
131072, from a single row (one generated token) to the rows of a training batch.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 1e-5
_IGNORE = -100
_NORM_MAX = 220000 * 512          # elements of the largest norm
_VOCAB_MAX = 4096 * 131072        # elements of the largest logits


def listed():
    return [
        # the norm in front of the gate for one generated token
        {"name": "norm_fwd_token", "op": "norm_fwd", "rows": 1, "cols": 4096, "dtype": "bf16",
         "wdtype": "bf16", "pad": 0},
        # the large-batch gate input of this library's own workload
        {"name": "norm_fwd_220k", "op": "norm_fwd", "rows": 220000, "cols": 512,
         "dtype": "bf16", "wdtype": "bf16", "pad": 0},
        # its training backward
        {"name": "norm_bwd_220k", "op": "norm_bwd", "rows": 220000, "cols": 512,
         "dtype": "bf16", "wdtype": "bf16", "pad": 0},
        # the LLM-sized gate input, 16-bit activations under fp32 norm weights
        {"name": "norm_bwd_llm", "op": "norm_bwd", "rows": 16384, "cols": 4096,
         "dtype": "fp16", "wdtype": "fp32", "pad": 0},
        # ragged batch, odd width, full precision
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 8191, "cols": 1023,
         "dtype": "fp32", "wdtype": "fp32", "pad": 0},
        # one generated token: its log probability and 20 alternatives
        {"name": "logprobs_token", "op": "logprobs", "rows": 1, "cols": 131072,
         "dtype": "bf16", "pad": 0, "top": 20, "temperature": 1.0, "masked": False},
        # a teacher's pass over a batch, its top 64 kept for the student
        {"name": "logprobs_teacher", "op": "logprobs", "rows": 4096, "cols": 131072,
         "dtype": "bf16", "pad": 0, "top": 64, "temperature": 1.0, "masked": False},
        # odd vocabulary with unusable entries masked, full precision
        {"name": "logprobs_odd", "op": "logprobs", "rows": 1021, "cols": 50021,
         "dtype": "fp32", "pad": 0, "top": 5, "temperature": 0.7, "masked": True},
        # policy-gradient step: gradient of log probability and entropy
        {"name": "logprobs_bwd", "op": "logprobs_bwd", "rows": 2048, "cols": 65536,
         "dtype": "bf16", "pad": 0, "top": 0, "temperature": 1.0, "masked": False},
        # distillation loss of a small validation batch
        {"name": "distill_fwd_small", "op": "distill_fwd", "rows": 37, "cols": 32000,
         "dtype": "fp16", "pad": 0, "top": 16, "temperature": 1.0},
        # distillation gradient, sliced out of a padded vocabulary
        {"name": "distill_bwd_odd", "op": "distill_bwd", "rows": 2047, "cols": 50021,
         "dtype": "bf16", "pad": 43, "top": 32, "temperature": 2.0},
        # a training step's loss and gradient
        {"name": "distill_step", "op": "distill_step", "rows": 4096, "cols": 131072,
         "dtype": "bf16", "pad": 0, "top": 64, "temperature": 2.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "logprobs", "logprobs_bwd", "distill_fwd",
                     "distill_bwd", "distill_step"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    pad = rng.choice([0, 0, 0, 1, 8, 43])
    if op.startswith("norm"):
        cols = _log_int(rng, 64, 14336)
        if rng.random() < 0.5:
            cols = max(64, cols // 8 * 8)
        budget = _NORM_MAX // (2 if dtype == "fp32" else 1)
        rows = _log_int(rng, 1, max(1, min(220000, budget // (cols + pad))))
        wdtype = "fp32" if dtype == "fp32" else rng.choice([dtype, "fp32"])
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "wdtype": wdtype,
                "pad": pad}
    cols = _log_int(rng, 500, 131072)
    if rng.random() < 0.5:
        cols = cols // 8 * 8
    # half of the largest: a drawn case may take any of the directions
    budget = _VOCAB_MAX // (4 if dtype == "fp32" else 2)
    rows = _log_int(rng, 1, max(1, min(8192, budget // (cols + pad))))
    case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "pad": pad,
            "top": rng.choice([0, 1, 5, 20, 64] if op.startswith("logprobs")
                              else [1, 8, 16, 50, 64]),
            "temperature": rng.choice([1.0, 0.7, 1.5] if op.startswith("logprobs")
                                      else [1.0, 2.0, 4.0])}
    if op.startswith("logprobs"):
        case["masked"] = rng.choice([False, True])
    return case


def _seeded(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _sliced(rows, cols, pad, dtype, g, scale):
    """Normal values [rows, cols] as a view into rows of cols + pad."""
    full = torch.randn(rows, cols + pad, dtype=dtype, device="cuda", generator=g)
    full *= scale
    return full[:, :cols]


def prepare(case, seed):
    g = _seeded(seed)
    R, C, dt = case["rows"], case["cols"], _DT[case["dtype"]]
    s = dict(case)
    if case["op"].startswith("norm"):
        wdt = _DT[case["wdtype"]]
        x = _sliced(R, C, case["pad"], dt, g, 1.0)
        # residual streams: a mean that differs by row, and a few channels that stand out
        x += torch.randn(R, 1, dtype=dt, device="cuda", generator=g) * 0.5
        x[:, ::97] *= 8.0
        s["x"] = x
        s["w"] = (1.0 + 0.2 * torch.randn(C, device="cuda", generator=g)).to(wdt)
        s["b"] = (0.1 * torch.randn(C, device="cuda", generator=g)).to(wdt)
        if case["op"] == "norm_fwd":
            s["y"] = torch.empty(R, C, dtype=dt, device="cuda")
            s["mean"] = torch.empty(R, device="cuda")
            s["rstd"] = torch.empty(R, device="cuda")
        else:
            s["dy"] = _sliced(R, C, 0, dt, g, 0.1)
            mean, rstd = [], []
            for c in x.split(16384):
                v, m = torch.var_mean(c.double(), dim=1, correction=0)
                mean.append(m)
                rstd.append((v + _EPS).rsqrt())
            s["mean"], s["rstd"] = torch.cat(mean).float(), torch.cat(rstd).float()
            s["dx"] = torch.empty(R, C, dtype=dt, device="cuda")
            s["dw"] = torch.empty(C, dtype=wdt, device="cuda")
            s["db"] = torch.empty(C, dtype=wdt, device="cuda")
        return s

    z = _sliced(R, C, case["pad"], dt, g, 2.0)
    T, k = case["temperature"], case["top"]
    if case["op"].startswith("logprobs"):
        # the token that was taken is mostly a likely one; it is never a masked one
        t = torch.randint(0, C, (R,), device="cuda", generator=g)
        if case["masked"]:
            z[:, 5::16] = -math.inf
            t = torch.where(t % 16 == 5, t - 1, t)
        lift = 6.0 + 2.0 * torch.randn(R, 1, device="cuda", generator=g)
        z.scatter_(1, t[:, None], lift.to(dt))
        if R >= 8:   # prompt and padding positions carry no target
            t[::8] = _IGNORE
        s["logits"], s["targets"] = z, t
        if case["op"] == "logprobs_bwd":
            lse, ent = [], []
            for c in z.split(max(1, (1 << 26) // C)):
                a = c.double() / T
                l = torch.logsumexp(a, 1, keepdim=True)
                p = torch.exp(a - l)
                ent.append(l[:, 0] - torch.where(p > 0, p * a, 0.0).sum(1))
                lse.append(l[:, 0])
            s["lse"], s["entropy"] = torch.cat(lse).float(), torch.cat(ent).float()
            s["dlogprob"] = torch.randn(R, device="cuda", generator=g)
            s["dentropy"] = torch.full((R,), -0.01, device="cuda")
            s["dlogits"] = torch.empty(R, C, dtype=dt, device="cuda")
        return s

    # the teacher's entries: distinct ids, one per stratum of the vocabulary, in falling order
    # of its logits; the student agrees with them up to noise
    u = torch.rand(R, k, device="cuda", generator=g)
    j = torch.arange(k, device="cuda")
    ids = ((j * C) // k + (u * (C // k)).long().clamp_(max=C // k - 1))
    ids = torch.gather(ids, 1, torch.rand(R, k, device="cuda", generator=g).argsort(1))
    top = 10.0 + 2.0 * torch.randn(R, k, device="cuda", generator=g)
    top = top.sort(1, descending=True).values
    near = top + torch.randn(R, k, device="cuda", generator=g)
    z.scatter_(1, ids, near.to(dt))
    if k >= 8:   # some rows kept fewer entries (a nucleus cut): the rest is padding
        ids[::3, k - 3:] = -1
    s["logits"], s["top_logits"], s["top_ids"] = z, top, ids
    if case["op"] == "distill_bwd":
        lse = [torch.logsumexp(c.double() / T, 1)
               for c in z.split(max(1, (1 << 26) // C))]
        s["lse"] = torch.cat(lse).float()
    if case["op"] != "distill_fwd":
        s["weight"] = (0.5 + torch.rand(R, device="cuda", generator=g)) / R
        s["dlogits"] = torch.empty(R, C, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms (fp32)
def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.sum(1, keepdim=True) / x.shape[1]
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / x.shape[1] + _EPS)
    y = d * rstd * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_bwd(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["w"].float()
    n = x.shape[1]
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    h = dy * w
    c1 = h.sum(1, keepdim=True) / n
    c2 = (h * xh).sum(1, keepdim=True) / n
    dx = rstd * (h - c1 - xh * c2)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return dx.to(s["x"].dtype), dw.to(s["w"].dtype), db.to(s["w"].dtype)


def _plain_lse(a):
    m = a.amax(1, keepdim=True)
    return m + torch.log(torch.exp(a - m).sum(1, keepdim=True))


def _plain_logprobs(s):
    z = s["logits"].float()
    C, k, t = z.shape[1], s["top"], s["targets"]
    a = z / s["temperature"]
    lse = _plain_lse(a)
    lp = a - lse
    p = torch.exp(lp)
    ent = -torch.where(p > 0, p * lp, 0.0).sum(1)
    taken = lp.gather(1, t.clamp(0, C - 1)[:, None])[:, 0]
    taken = torch.where(t == _IGNORE, 0.0, taken)
    if k == 0:
        return taken, ent, lse[:, 0]
    # largest first, equal ones by rising index: whole numbers that order the same way
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    order = order * C + torch.arange(C - 1, -1, -1, device=z.device)
    ids = torch.topk(order, k, dim=1, sorted=True).indices
    return taken, ent, lse[:, 0], lp.gather(1, ids), ids


def _plain_logprobs_bwd(s):
    z, t, T = s["logits"].float(), s["targets"], s["temperature"]
    C = z.shape[1]
    lp = z / T - s["lse"][:, None]
    p = torch.exp(lp)
    g = torch.where(t == _IGNORE, 0.0, s["dlogprob"])[:, None]
    h = s["dentropy"][:, None]
    da = -g * p - torch.where(p > 0, h * p * (lp + s["entropy"][:, None]), 0.0)
    da.scatter_add_(1, t.clamp(0, C - 1)[:, None], g)
    return (da / T).to(s["logits"].dtype)


def _plain_teacher(s):
    ids, T = s["top_ids"], s["temperature"]
    C = s["logits"].shape[1]
    u = torch.where((ids >= 0) & (ids < C), s["top_logits"].float() / T, -math.inf)
    lq = u - _plain_lse(u)
    return lq, torch.exp(lq), ids.clamp(0, C - 1)


def _plain_distill_fwd(s):
    T = s["temperature"]
    lq, q, ids = _plain_teacher(s)
    a = s["logits"].float() / T
    lse = _plain_lse(a)
    lp = a.gather(1, ids) - lse
    loss = T * T * torch.where(q > 0, q * (lq - lp), 0.0).sum(1)
    return loss, lse[:, 0]


def _plain_distill_bwd(s, lse):
    T = s["temperature"]
    _, q, ids = _plain_teacher(s)
    d = torch.exp(s["logits"].float() / T - lse[:, None])
    d.scatter_add_(1, ids, -q)
    return (d * (s["weight"] * T)[:, None]).to(s["logits"].dtype)


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "logprobs":
        return _plain_logprobs(s)
    if op == "logprobs_bwd":
        return _plain_logprobs_bwd(s)
    if op == "distill_fwd":
        return _plain_distill_fwd(s)
    if op == "distill_bwd":
        return _plain_distill_bwd(s, s["lse"])
    loss, lse = _plain_distill_fwd(s)
    return loss, _plain_distill_bwd(s, lse)


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import swish_activation_backward_amd as swg
    op = s["op"]
    if op == "norm_fwd":
        return swg.layer_norm_fwd(s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"],
                                  eps=_EPS)
    if op == "norm_bwd":
        swg.layer_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"],
                           s["db"])
        return s["dx"], s["dw"], s["db"]
    T = s["temperature"]
    if op == "logprobs":
        r = swg.token_logprobs(s["logits"], s["targets"], top=s["top"], temperature=T,
                               ignore_index=_IGNORE)
        if s["top"] == 0:
            return r.logprob, r.entropy, r.lse
        return r.logprob, r.entropy, r.lse, r.top_logprob, r.top_id
    if op == "logprobs_bwd":
        return swg.token_logprobs_bwd(s["logits"], s["targets"], s["lse"], s["entropy"],
                                      s["dlogprob"], s["dentropy"], s["dlogits"],
                                      temperature=T, ignore_index=_IGNORE)
    if op == "distill_fwd":
        return swg.distill_fwd(s["logits"], s["top_logits"], s["top_ids"], temperature=T)
    if op == "distill_bwd":
        return swg.distill_bwd(s["logits"], s["top_logits"], s["top_ids"], s["lse"],
                               s["weight"], s["dlogits"], temperature=T)
    loss, _, dlogits = swg.distill_fwd_bwd(s["logits"], s["top_logits"], s["top_ids"],
                                           s["weight"], s["dlogits"], temperature=T)
    return loss, dlogits


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot avoid
def work(case):
    R, C, es = case["rows"], case["cols"], _ES[case["dtype"]]
    n = R * C
    op = case["op"]
    if op.startswith("norm"):
        ws = _ES[case["wdtype"]]
        if op == "norm_fwd":
            return {"bytes": 2 * n * es + 2 * C * ws + 8 * R, "flops": 8 * n}
        return {"bytes": 3 * n * es + 3 * C * ws + 8 * R, "flops": 16 * n}
    k = case["top"]
    if op == "logprobs":
        return {"bytes": n * es + R * (8 + 12 + 12 * k), "flops": 6 * n}
    if op == "logprobs_bwd":
        return {"bytes": 2 * n * es + R * (8 + 16), "flops": 8 * n}
    teacher = R * k * (4 + 8)
    if op == "distill_fwd":
        return {"bytes": n * es + teacher + 8 * R, "flops": 4 * n}
    if op == "distill_bwd":
        return {"bytes": 2 * n * es + teacher + 8 * R, "flops": 4 * n}
    return {"bytes": 2 * n * es + teacher + 8 * R, "flops": 8 * n}


# ------------------------------------------------------------------ the definitions in float64
def _chunks(n_rows, cols, limit=1 << 25):
    step = max(1, limit // cols)
    return [slice(i, min(n_rows, i + step)) for i in range(0, n_rows, step)]


def _exact_norm(s):
    x, w, b = s["x"], s["w"].double(), s["b"].double()
    R, C = x.shape
    fwd = s["op"] == "norm_fwd"
    rows = []
    dw = torch.zeros(C, dtype=torch.float64, device=x.device)
    db = torch.zeros_like(dw)
    for c in _chunks(R, C):
        xd = x[c].double()
        if fwd:
            var, mean = torch.var_mean(xd, dim=1, keepdim=True, correction=0)
            rstd = (var + _EPS) ** -0.5
            rows.append(((xd - mean) * rstd * w + b, mean[:, 0], rstd[:, 0]))
            continue
        mu, r = s["mean"][c, None].double(), s["rstd"][c, None].double()
        dy = s["dy"][c].double()
        xh = (xd - mu) * r
        # dx = rstd (I - 1 1'/C - xh xh'/C) (dy w)
        v = dy * w
        along = torch.linalg.vecdot(v, xh)[:, None] / C
        rows.append((r * (v - v.mean(1, keepdim=True) - xh * along),))
        dw += torch.einsum("rc,rc->c", dy, xh)
        db += dy.sum(0)
    out = tuple(torch.cat(t) for t in zip(*rows))
    return out if fwd else (out[0], dw, db)


def _exact_vocab(s):
    z, T, op, k = s["logits"], s["temperature"], s["op"], s["top"]
    R, C = z.shape
    rows = []
    for c in _chunks(R, C):
        zc = z[c].double()
        logp = torch.log_softmax(zc / T, dim=1)
        lse = torch.logsumexp(zc / T, dim=1)
        p = logp.exp()
        n = torch.arange(zc.shape[0], device=z.device)
        if op.startswith("logprobs"):
            t = s["targets"][c]
            live = t != _IGNORE
            tt = t.clamp(min=0)
            if op == "logprobs":
                ent = torch.special.entr(p).sum(1)
                row = (torch.where(live, logp[n, tt], 0.0), ent, lse)
                if k:
                    ids = torch.sort(zc, dim=1, descending=True, stable=True).indices[:, :k]
                    row += (logp.gather(1, ids), ids)
            else:
                logp = zc / T - s["lse"][c, None].double()
                p = logp.exp()
                ent = s["entropy"][c, None].double()
                g = s["dlogprob"][c].double() * live
                d = -p * g[:, None]
                d[n, tt] += g
                d += s["dentropy"][c, None].double() * (torch.special.entr(p) - p * ent)
                row = (d / T,)
        else:
            ids = s["top_ids"][c]
            keep = ids >= 0
            u = (s["top_logits"][c].double() / T).masked_fill(~keep, -math.inf)
            q = torch.softmax(u, 1)
            at = ids.clamp(min=0)
            row = ()
            if op != "distill_bwd":
                kl = -torch.special.entr(q) - torch.special.xlogy(q, p.gather(1, at))
                row += (T * T * kl.sum(1),)
            if op == "distill_fwd":
                row += (lse,)
            else:
                if op == "distill_bwd":
                    p = torch.exp(zc / T - s["lse"][c, None].double())
                soft = torch.zeros_like(p).scatter_add_(1, at, q)
                row += (T * s["weight"][c, None].double() * (p - soft),)
        rows.append(row)
    out = tuple(torch.cat(t) for t in zip(*rows))
    return out[0] if len(out) == 1 else out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"].startswith("norm") else _exact_vocab(s)
