"""Timed cases of the output layer's token log-probabilities and distillation.

Five operators over the logits: the log-probability of a given token in each
row with the row's entropy, the token's rank and the most likely alternatives
(`logprobs`) and its gradient (`logprobs_bwd`); and the cross-entropy against a
teacher that is known by its top tokens only (`distill_fwd`, `distill_bwd`, and
both in one call, `distill_fused`).  `run` computes them either in a plain form
in elementary torch operations or, with `own` set, through this package's entry
points.
"""
import math

import torch

own = False  # True: the package's kernels; False: the plain forms


def _package():
    import lm_head_fp32_amd as lmh

    return lmh


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # One request's next token with five alternatives: latency.
        {"name": "logprobs_token", "op": "logprobs", "n": 1, "V": 32768, "dtype": "fp32", "top": 5,
         "rank": True, "temperature": "rows"},
        # A decode batch that returns twenty alternatives per token, BF16 logits.
        {"name": "logprobs_decode_64", "op": "logprobs", "n": 64, "V": 131072, "dtype": "bf16", "top": 20,
         "rank": True, "temperature": "rows"},
        # A prompt's tokens, odd length and vocabulary.
        {"name": "logprobs_prompt_odd", "op": "logprobs", "n": 777, "V": 50001, "dtype": "fp32", "top": 10,
         "rank": True, "temperature": "none"},
        # Scoring of sampled sequences for a policy gradient: no alternatives.
        {"name": "logprobs_rollout", "op": "logprobs", "n": 8192, "V": 131072, "dtype": "fp32", "top": 0,
         "rank": False, "temperature": "one"},
        # Policy gradient with an entropy bonus, a small odd batch of BF16 logits.
        {"name": "logprobs_bwd_odd", "op": "logprobs_bwd", "n": 101, "V": 32003, "dtype": "bf16",
         "grad": "bf16", "entropy": True, "temperature": "none"},
        # The same over a training batch.
        {"name": "logprobs_bwd_train", "op": "logprobs_bwd", "n": 4096, "V": 131072, "dtype": "fp32",
         "grad": "bf16", "entropy": True, "temperature": "one"},
        # Evaluation of a small odd batch against lists of up to sixteen log-probabilities.
        {"name": "distill_fwd_odd", "op": "distill_fwd", "n": 33, "V": 32003, "dtype": "fp32", "k": 16,
         "values": "bf16", "tail": True, "ragged": True, "temperature": "none"},
        # Evaluation over a large vocabulary, the teacher's 64 largest logits.
        {"name": "distill_fwd_eval", "op": "distill_fwd", "n": 1024, "V": 131072, "dtype": "fp32", "k": 64,
         "values": "fp32", "tail": False, "ragged": False, "temperature": "one"},
        # Gradient alone, an odd batch, FP32 out.
        {"name": "distill_bwd_odd", "op": "distill_bwd", "n": 129, "V": 50001, "dtype": "fp32", "k": 20,
         "values": "fp32", "tail": False, "ragged": True, "temperature": "one", "grad": "fp32"},
        # Gradient of a batch over a large vocabulary, with the rest of the vocabulary as one class.
        {"name": "distill_bwd_train", "op": "distill_bwd", "n": 2048, "V": 131072, "dtype": "fp32", "k": 64,
         "values": "fp32", "tail": True, "ragged": False, "temperature": "none", "grad": "bf16"},
        # Loss and gradient together: a small step.
        {"name": "distill_fused_128", "op": "distill_fused", "n": 128, "V": 32768, "dtype": "fp32", "k": 32,
         "values": "fp32", "tail": False, "ragged": True, "temperature": "one", "grad": "bf16"},
        # Loss and gradient together: the training step's batch.
        {"name": "distill_fused_train", "op": "distill_fused", "n": 1024, "V": 32768, "dtype": "fp32",
         "k": 64, "values": "bf16", "tail": True, "ragged": False, "temperature": "none", "grad": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_bwd", "distill_fwd", "distill_bwd", "distill_fused"])
    V = _log_uniform(rng, 1000, 131072)
    case = {"op": op, "V": V, "dtype": rng.choice(["fp32", "fp32", "bf16"]),
            "temperature": rng.choice(["none", "one", "rows"])}
    most = 2 ** 28  # logits
    if op == "logprobs":
        case["top"] = rng.choice([0, 0, 1, 5, 20, 64])
        case["rank"] = rng.choice([True, False])
        most = 2 ** 25 if case["top"] else 2 ** 29
    elif op == "logprobs_bwd":
        case["entropy"] = rng.choice([True, False])
    else:
        case["k"] = _log_uniform(rng, 1, 128)
        case["values"] = rng.choice(["fp32", "bf16"])
        case["tail"] = rng.choice([True, False])
        case["ragged"] = rng.choice([True, False])
    if op not in ("logprobs", "distill_fwd"):
        case["grad"] = rng.choice(["bf16", "bf16", "fp32"])
    case["n"] = _log_uniform(rng, 1, min(8192, most // V))
    return case


_TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _rows(shape, dtype):
    """A tensor whose rows start at 16-byte boundaries, as the package's own
    outputs do."""
    mult = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = (shape[-1] + mult - 1) // mult * mult
    return torch.zeros(*shape[:-1], ld, dtype=dtype, device="cuda")[..., : shape[-1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, V, op = case["n"], case["V"], case["op"]

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    s = {"op": op, "case": case}
    z = _rows((n, V), torch.float32)
    z.normal_(0.0, 3.0, generator=gen)
    at = torch.randint(0, V, (n, 1), device="cuda", generator=gen)
    # what a trained model is fairly sure of
    z.scatter_add_(1, at, torch.where(uniform(n, 1) < 0.7, 10.0 * uniform(n, 1) + 4.0, 0.0))
    kind = case["temperature"]
    s["temperature"] = (None if kind == "none" else 1.0 + uniform(1) if kind == "one"
                        else 0.6 + 0.8 * uniform(n))
    if op in ("logprobs", "logprobs_bwd"):
        # one token in sixteen belongs to a prompt or to padding
        s["token"] = torch.where(uniform(n) < 1.0 / 16, -100, at[:, 0]).to(torch.int32)
    else:
        k = case["k"]
        # the teacher: the student's logits in part, and an opinion of its own
        t = _rows((n, V), torch.float32)
        t.normal_(0.0, 1.5, generator=gen)
        t += 0.75 * z
        best, where = torch.topk(t, k, dim=1)
        if case["tail"]:
            T = 1.0 if s["temperature"] is None else s["temperature"].reshape(-1, 1)
            best = best / T - torch.logsumexp(t / T, 1, keepdim=True)
        del t
        if case["ragged"]:
            length = torch.randint(0, k + 1, (n, 1), device="cuda", generator=gen)
            absent = torch.arange(k, device="cuda")[None, :] >= length
            where = torch.where(absent, -1, where)
            best = torch.where(absent, -math.inf, best)
        s["t_token"] = where.to(torch.int32).contiguous()
        s["t_value"] = best.to(_TORCH[case["values"]]).contiguous()
    if case["dtype"] == "bf16":
        s["logits"] = _rows((n, V), torch.bfloat16)
        s["logits"].copy_(z)
    else:
        s["logits"] = z
    del z
    # upstream gradients: advantages over the rows' count; a constant bonus
    if op == "logprobs_bwd":
        s["d_logprob"] = torch.randn(n, device="cuda", generator=gen) / n
        s["d_entropy"] = torch.full((1,), -0.01 / n, device="cuda") if case["entropy"] else None
        s["stats"] = _plain_logprobs(s)["stats"]
    elif op in ("distill_bwd", "distill_fused"):
        s["d_loss"] = torch.full((1,), 1.0 / n, device="cuda")
        if op == "distill_bwd":
            s["stats"] = _plain_distill_fwd(s)["stats"]
    return s


# ----------------------------------------------------------------------- run

def run(s):
    op, c = s["op"], s["case"]
    if own:
        lmh = _package()
        if op == "logprobs":
            got = lmh.lmhead_logprobs(s["logits"], s["token"], temperature=s["temperature"], n_top=c["top"],
                                      rank=None if c["rank"] else False)
            names = ("logprob", "entropy", "rank", "top_logprob", "top_token", "stats")
            return {k: v for k, v in zip(names, got) if v is not None}
        if op == "logprobs_bwd":
            return lmh.lmhead_logprobs_bwd(s["logits"], s["stats"], s["token"], s["d_logprob"],
                                           dentropy=s["d_entropy"], temperature=s["temperature"],
                                           grad_dtype=c["grad"])
        teacher = (s["t_token"], s["t_value"])
        how = {"tail": c["tail"], "temperature": s["temperature"]}
        if op == "distill_fwd":
            loss, stats = lmh.lmhead_distill_fwd(s["logits"], *teacher, **how)
            return {"loss": loss, "stats": stats}
        if op == "distill_bwd":
            return lmh.lmhead_distill_bwd(s["logits"], s["stats"], *teacher, s["d_loss"],
                                          grad_dtype=c["grad"], **how)
        loss, stats, g = lmh.lmhead_distill_fused(s["logits"], *teacher, s["d_loss"], grad_dtype=c["grad"],
                                                  **how)
        return {"loss": loss, "stats": stats, "dlogits": g}
    if op == "logprobs":
        return _plain_logprobs(s)
    if op == "logprobs_bwd":
        return _plain_logprobs_bwd(s)
    if op == "distill_fwd":
        return _plain_distill_fwd(s)
    if op == "distill_bwd":
        return _plain_distill_bwd(s, s["stats"])
    out = _plain_distill_fwd(s)
    out["dlogits"] = _plain_distill_bwd(s, out["stats"])
    return out


def _inverse_temperature(s):
    return 1.0 if s["temperature"] is None else 1.0 / s["temperature"].reshape(-1, 1)


def _plain_logprobs(s):
    c = s["case"]
    z = s["logits"].float()
    V = z.shape[1]
    m = z.amax(1, keepdim=True)
    x = (z - m) * _inverse_temperature(s)
    e = torch.exp(x)
    d = e.sum(1, keepdim=True)
    log_d = torch.log(d)
    entropy = log_d - (e * x).sum(1, keepdim=True) / d
    y = s["token"].long()[:, None]
    given = y >= 0
    at = y.clamp(min=0)
    logprob = torch.where(given, torch.gather(x, 1, at) - log_d, 0.0)
    out = {"logprob": logprob[:, 0], "entropy": entropy[:, 0]}
    if c.get("rank"):
        own_z = torch.gather(z, 1, at)
        ahead = (z > own_z) | ((z == own_z) & (torch.arange(V, device="cuda")[None, :] < at))
        out["rank"] = torch.where(given[:, 0], ahead.sum(1), -1).to(torch.int32)
    if c.get("top"):
        _, idx = torch.sort(z, dim=1, descending=True, stable=True)
        idx = idx[:, : c["top"]]
        out["top_logprob"] = torch.gather(x, 1, idx) - log_d
        out["top_token"] = idx.to(torch.int32)
    out["stats"] = torch.cat([m, d, entropy, logprob], 1)
    return out


def _plain_logprobs_bwd(s):
    c = s["case"]
    z, st = s["logits"].float(), s["stats"]
    inv_t = _inverse_temperature(s)
    m, d, entropy = st[:, 0:1], st[:, 1:2], st[:, 2:3]
    x = (z - m) * inv_t
    p = torch.exp(x) / d
    y = s["token"].long()[:, None]
    given = y >= 0
    g = torch.where(given, s["d_logprob"][:, None], 0.0)
    out = -g * p
    if s["d_entropy"] is not None:
        out = out - s["d_entropy"] * p * (x - torch.log(d) + entropy)
    out.scatter_add_(1, y.clamp(min=0), g)
    return (out * inv_t).to(_TORCH[c["grad"]])


def _teacher(s):
    """(q, shift, sum) of the listed tokens, their columns and which are there."""
    there = s["t_token"] >= 0
    v = s["t_value"].float()
    if s["case"]["tail"]:
        q = torch.where(there, torch.exp(v), 0.0)
        top, total = torch.zeros_like(v[:, :1]), torch.ones_like(v[:, :1])
    else:
        top = torch.where(there, v, -math.inf).amax(1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        e = torch.where(there, torch.exp((v - top) * _inverse_temperature(s)), 0.0)
        total = e.sum(1, keepdim=True)
        q = e / total.clamp(min=1e-30)
    return q, top, total, s["t_token"].long().clamp(min=0), there


def _plain_distill_fwd(s):
    z = s["logits"].float()
    inv_t = _inverse_temperature(s)
    q, top, total, at, there = _teacher(s)
    held = there.any(1, keepdim=True)
    m = z.amax(1, keepdim=True)
    e = torch.exp((z - m) * inv_t)
    d = e.sum(1, keepdim=True)
    logp = (torch.gather(z, 1, at) - m) * inv_t - torch.log(d)
    # differences of near-equal numbers: in 64 bits
    q64 = q.double()
    terms = torch.where(q > 0, q64 * (torch.log(q64) - logp.double()), 0.0)
    loss = terms.sum(1, keepdim=True)
    weight = q64.sum(1, keepdim=True)
    other, w = m, weight / d
    if s["case"]["tail"]:
        taken = torch.zeros_like(z).scatter_add_(1, at, there.float()) > 0
        zr = torch.where(taken, -math.inf, z)
        other = zr.amax(1, keepdim=True)
        rest = torch.exp((zr - other) * inv_t).sum(1, keepdim=True).double()
        q_rest = (1.0 - weight).clamp(min=0.0)
        scale = torch.exp((other - m).double() * inv_t)
        log_p = (other - m).double() * inv_t + torch.log(rest) - torch.log(d.double())
        loss = loss + torch.where(q_rest > 0, q_rest * (torch.log(q_rest) - log_p), 0.0)
        weight = weight + q_rest
        w = weight * scale / d - q_rest / rest
    loss = torch.where(held, loss, 0.0).float()
    stats = torch.cat([m, d, loss, weight.float(), other, w.float(), top, total], 1)
    return {"loss": loss[:, 0], "stats": torch.where(held, stats, 0.0)}


def _plain_distill_bwd(s, stats):
    z = s["logits"].float()
    inv_t = _inverse_temperature(s)
    q, _, _, at, there = _teacher(s)
    m, d, _, weight, other, w, _, _ = (stats[:, i: i + 1] for i in range(8))
    held = there.any(1, keepdim=True)
    out = torch.exp((z - other) * inv_t) * w
    listed_grad = torch.exp((torch.gather(z, 1, at) - m) * inv_t) * (weight / d.clamp(min=1e-30)) - q
    V = z.shape[1]
    out = torch.cat([out, torch.zeros_like(m)], 1)  # a column for what is absent
    out.scatter_(1, torch.where(there, at, V), listed_grad)
    out = torch.where(held, out[:, :V] * (s["d_loss"] * inv_t), 0.0)
    return out.to(_TORCH[s["case"]["grad"]])


# ---------------------------------------------------------------- exact, work

def _chunks(case):
    step = max(1, 2 ** 26 // case["V"])
    return [(r, min(r + step, case["n"])) for r in range(0, case["n"], step)]


def _exact_logprobs(s, lo, hi):
    c = s["case"]
    z = s["logits"][lo:hi].double()
    T = torch.ones(hi - lo, 1, dtype=torch.float64, device="cuda")
    if s["temperature"] is not None:
        T = s["temperature"].double().expand(c["n"])[lo:hi, None]
    x = z / T
    lse = torch.logsumexp(x, 1, keepdim=True)
    lp = x - lse
    m = z.amax(1, keepdim=True)
    y = s["token"][lo:hi].long()
    rows = torch.arange(hi - lo, device="cuda")
    given = y >= 0
    chosen = torch.where(given, lp[rows, y.clamp(min=0)], 0.0)
    entropy = -(torch.exp(lp) * lp).sum(1)
    if s["op"] == "logprobs_bwd":
        p = torch.exp(lp)
        one_hot = torch.zeros_like(p)
        one_hot[rows[given], y[given]] = 1.0
        g = torch.where(given, s["d_logprob"][lo:hi].double(), 0.0)[:, None]
        out = g * (one_hot - p)
        if s["d_entropy"] is not None:
            out = out - s["d_entropy"].double() * p * (lp + entropy[:, None])
        return {"dlogits": out / T}
    out = {"logprob": chosen, "entropy": entropy}
    if c["rank"]:
        kept = torch.full_like(y, -1)
        for i in torch.nonzero(given).flatten().tolist():
            own_z = z[i, y[i]]
            kept[i] = (z[i] > own_z).sum() + (z[i, : y[i]] == own_z).sum()
        out["rank"] = kept.to(torch.int32)
    if c["top"]:
        tops, ids = [], []
        for i in range(hi - lo):
            kth = torch.topk(z[i], c["top"]).values[-1]
            cand = torch.nonzero(z[i] >= kth).flatten()
            order = sorted(zip((-z[i, cand]).tolist(), cand.tolist()))[: c["top"]]
            ids.append([j for _, j in order])
            tops.append(lp[i, ids[-1]])
        out["top_logprob"] = torch.stack(tops)
        out["top_token"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
    out["stats"] = torch.stack([m[:, 0], torch.exp(lse - m / T)[:, 0], entropy, chosen], 1)
    return out


def _exact_distill(s, lo, hi):
    c = s["case"]
    z = s["logits"][lo:hi].double()
    n, V = z.shape
    T = torch.ones(n, 1, dtype=torch.float64, device="cuda")
    if s["temperature"] is not None:
        T = s["temperature"].double().expand(c["n"])[lo:hi, None]
    x = z / T
    lse = torch.logsumexp(x, 1, keepdim=True)
    lp = x - lse
    ids, v = s["t_token"][lo:hi].long(), s["t_value"][lo:hi].double()
    r, j = torch.nonzero(ids >= 0, as_tuple=True)
    held = (ids >= 0).any(1)
    # the teacher laid out over the whole vocabulary
    logq = torch.full((n, V), -math.inf, dtype=torch.float64, device="cuda")
    logq[r, ids[r, j]] = v[r, j] if c["tail"] else v[r, j] / T[r, 0]
    if not c["tail"]:
        norm = torch.where(held[:, None], torch.logsumexp(logq, 1, keepdim=True), 0.0)
        logq = logq - norm
    there = logq > -math.inf
    q = torch.exp(logq)
    loss = torch.where(there, q * (logq - lp), 0.0).sum(1)
    total = q.sum(1)
    if c["tail"]:
        rest = torch.where(there, -math.inf, lp)
        log_rest = torch.logsumexp(rest, 1)
        q_rest = (1.0 - total).clamp(min=0.0)
        loss = loss + torch.where(q_rest > 0, q_rest * (torch.log(q_rest) - log_rest), 0.0)
        total = total + q_rest
    out = {}
    if s["op"] != "distill_bwd":
        m = z.amax(1)
        d = torch.exp(lse - m[:, None] / T)[:, 0]
        other, w = m, total / d
        top = torch.zeros(n, dtype=torch.float64, device="cuda")
        t_sum = torch.ones_like(top)
        if c["tail"]:
            other = torch.where(there, -math.inf, z).amax(1)
            # p / exp((z - other) / T), the same for every column
            unit = torch.exp(other / T[:, 0] - lse[:, 0])
            w = unit * total - q_rest * unit / torch.exp(log_rest)
        else:
            top = torch.where(ids >= 0, v, -math.inf).amax(1)
            t_sum = torch.exp(norm[:, 0] - top / T[:, 0])
        stats = torch.stack([m, d, loss, total, other, w, top, t_sum], 1)
        out["loss"] = torch.where(held, loss, 0.0)
        out["stats"] = torch.where(held[:, None], stats, 0.0)
    if s["op"] != "distill_fwd":
        p = torch.exp(lp)
        g = total[:, None] * p - q
        if c["tail"]:
            g = g - torch.where(there, 0.0, q_rest[:, None] * torch.exp(lp - log_rest[:, None]))
        g = torch.where(held[:, None], g * s["d_loss"].double() / T, 0.0)
        out["dlogits"] = g
    return out


def exact(case, seed):
    """The definitions in 64 bits, over the whole vocabulary."""
    s = prepare(case, seed)
    f = _exact_logprobs if case["op"].startswith("logprobs") else _exact_distill
    parts = [f(s, lo, hi) for lo, hi in _chunks(case)]
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return out["dlogits"] if case["op"].endswith("_bwd") else out


def work(case):
    n, V = case["n"], case["V"]
    size = {"fp32": 4, "bf16": 2}
    read = n * V * size[case["dtype"]]
    if case["op"].startswith("logprobs"):
        if case["op"] == "logprobs":
            return {"bytes": read + n * (4 + 8 + 16 + 4 * case["rank"] + 8 * case["top"]),
                    "flops": 6.0 * n * V}
        return {"bytes": read + n * V * size[case["grad"]] + n * 24, "flops": (7.0 if case["entropy"] else 4.0) * n * V}
    lists = n * case["k"] * (4 + size[case["values"]])
    if case["op"] == "distill_fwd":
        return {"bytes": read + lists + n * 36, "flops": 4.0 * n * V}
    flops = 4.0 if case["op"] == "distill_bwd" else 5.0
    return {"bytes": read + n * V * size[case["grad"]] + lists + n * 36, "flops": flops * n * V}
