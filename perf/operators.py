"""Timed cases of the output layer's adapter and beam-search operators.

Four operators: the logits of a batch whose tokens use different low-rank
adapters beside the shared vocabulary weight (`logits_lora`), the gradients of
such adapters (`lora_bwd`), the selection of the next beams from the logits
(`beam_select`) and the reordering of per-beam states that follows it
(`beam_reorder`).  `run` computes them either in a plain form in elementary
torch operations or, with `own` set, through this package's entry points.
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
        # One sequence's next token, one adapter: the smallest decode step, bound by W.
        {"name": "logits_lora_token", "op": "logits_lora", "M": 1, "K": 4096, "V": 32768, "r": 16,
         "n": 8, "order": "mixed", "out": "fp32"},
        # A decode batch of 128 requests spread over 32 adapters, some on none.
        {"name": "logits_lora_decode_128", "op": "logits_lora", "M": 128, "K": 4096, "V": 32768,
         "r": 16, "n": 32, "order": "mixed", "out": "fp32"},
        # An odd decode batch, vocabulary and rank, BF16 logits.
        {"name": "logits_lora_odd", "op": "logits_lora", "M": 37, "K": 2040, "V": 32003, "r": 12,
         "n": 5, "order": "mixed", "out": "bf16"},
        # A prefill or training batch: four requests' runs of tokens, a larger rank.
        {"name": "logits_lora_prefill", "op": "logits_lora", "M": 1024, "K": 8192, "V": 32768,
         "r": 64, "n": 4, "order": "runs", "out": "fp32"},
        # Gradients of a small batch over a few adapters, odd row count and vocabulary.
        {"name": "lora_bwd_small", "op": "lora_bwd", "M": 101, "K": 4096, "V": 32003, "r": 8, "n": 3,
         "order": "mixed"},
        # Gradients of the training batch, four adapters.
        {"name": "lora_bwd_train", "op": "lora_bwd", "M": 1024, "K": 8192, "V": 32768, "r": 16,
         "n": 4, "order": "runs"},
        # One request with four beams: latency.
        {"name": "beam_select_1x4", "op": "beam_select", "B": 1, "W": 4, "V": 32768, "out_beams": 4,
         "dtype": "fp32", "finished": 0.0},
        # Odd vocabulary, BF16 logits, twice as many candidates as beams, a fifth of the beams ended.
        {"name": "beam_select_odd", "op": "beam_select", "B": 17, "W": 5, "V": 50001,
         "out_beams": 10, "dtype": "bf16", "finished": 0.2},
        # A full serving batch over a large vocabulary.
        {"name": "beam_select_64x8", "op": "beam_select", "B": 64, "W": 8, "V": 131072,
         "out_beams": 8, "dtype": "fp32", "finished": 0.1},
        # The tokens that four beams have written so far: latency.
        {"name": "beam_reorder_tokens", "op": "beam_reorder", "B": 1, "W": 4, "layers": 1, "heads": 1,
         "T": 512, "D": 1, "dtype": "int32", "ragged": False},
        # One layer's keys of an odd batch, ragged live lengths.
        {"name": "beam_reorder_ragged", "op": "beam_reorder", "B": 7, "W": 5, "layers": 2, "heads": 3,
         "T": 777, "D": 72, "dtype": "bf16", "ragged": True},
        # Keys and values of eight layers for 16 requests of four beams.
        {"name": "beam_reorder_cache", "op": "beam_reorder", "B": 16, "W": 4, "layers": 16, "heads": 8,
         "T": 1024, "D": 64, "dtype": "bf16", "ragged": True},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logits_lora", "lora_bwd", "beam_select", "beam_reorder"])
    if op in ("logits_lora", "lora_bwd"):
        r = rng.choice([4, 8, 12, 16, 24, 32, 64] if op == "logits_lora" else [4, 8, 12, 16])
        case = {"op": op, "M": _log_uniform(rng, 1, 1024), "K": 8 * _log_uniform(rng, 64, 1024),
                "V": _log_uniform(rng, 1000, 32768), "r": r,
                "n": _log_uniform(rng, 1, 256 // r if op == "logits_lora" else 4),
                "order": rng.choice(["mixed", "runs"])}
        if op == "logits_lora":
            case["out"] = rng.choice(["fp32", "fp32", "bf16"])
        return case
    if op == "beam_select":
        W = rng.randint(1, 8)
        return {"op": op, "B": _log_uniform(rng, 1, 64), "W": W, "V": _log_uniform(rng, 1000, 131072),
                "out_beams": rng.choice([W, 2 * W, 8]), "dtype": rng.choice(["fp32", "fp32", "bf16"]),
                "finished": rng.choice([0.0, 0.1, 0.3])}
    dtype = rng.choice(["bf16", "fp32", "int32"])
    return {"op": op, "B": _log_uniform(rng, 1, 16), "W": rng.randint(1, 4),
            "layers": _log_uniform(rng, 1, 16), "heads": rng.randint(1, 8),
            "T": _log_uniform(rng, 32, 1024), "D": rng.choice([1, 33, 40, 64] if dtype == "bf16" else [1, 17, 20, 32]),
            "dtype": dtype, "ragged": rng.choice([True, False])}


_TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32}


def _rows(shape, dtype):
    """An uninitialised tensor whose rows start at 16-byte boundaries, as the
    package's own outputs do."""
    mult = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = (shape[-1] + mult - 1) // mult * mult
    return torch.zeros(*shape[:-1], ld, dtype=dtype, device="cuda")[..., : shape[-1]]


def _normal(gen, shape, sigma, dtype):
    t = _rows(shape, dtype)
    t.copy_(torch.randn(*shape, device="cuda", generator=gen) * sigma)
    return t


def _adapters(gen, M, n, order):
    """Adapter of each token: every adapter in use where there are tokens
    enough, and about one token in sixteen on none."""
    ids = torch.arange(M, device="cuda") % n
    if order == "mixed":
        ids = ids[torch.randperm(M, device="cuda", generator=gen)]
    else:
        ids = ids.sort().values
    none = torch.rand(M, device="cuda", generator=gen) < 1.0 / 16
    return torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op in ("logits_lora", "lora_bwd"):
        M, K, V, r, n = (case[k] for k in ("M", "K", "V", "r", "n"))
        s["x"] = _normal(gen, (M, K), 1.0, torch.bfloat16)
        s["A"] = _normal(gen, (n, r, K), K ** -0.5, torch.bfloat16)
        s["B"] = _normal(gen, (n, V, r), 0.1, torch.bfloat16)
        s["scale"] = (1.0 + torch.rand(n, device="cuda", generator=gen)) * (16.0 / r)
        s["adapter"] = _adapters(gen, M, n, case["order"])
        if op == "logits_lora":
            s["W"] = _normal(gen, (V, K), 0.02, torch.bfloat16)
        else:
            # (softmax - one hot) / rows, as the cross-entropy backward writes it
            z = 3.0 * torch.randn(M, V, device="cuda", generator=gen)
            p = torch.exp(z - z.amax(1, keepdim=True))
            p /= p.sum(1, keepdim=True)
            y = torch.randint(0, V, (M, 1), device="cuda", generator=gen)
            p.scatter_add_(1, y, torch.full((M, 1), -1.0, device="cuda"))
            s["g"] = _rows((M, V), torch.bfloat16)
            s["g"].copy_(p / M)
    elif op == "beam_select":
        B, W, V = case["B"], case["W"], case["V"]
        s["logits"] = _normal(gen, (B * W, V), 3.0, _TORCH[case["dtype"]])
        s["scores"] = -40.0 + 2.0 * torch.randn(B, W, device="cuda", generator=gen)
        s["finished"] = torch.rand(B, W, device="cuda", generator=gen) < case["finished"]
        s["eos"] = V - 1
    else:
        B, W, D = case["B"], case["W"], case["D"]
        shape = (case["layers"], B * W, case["heads"], case["T"], D)
        dt = _TORCH[case["dtype"]]
        for name in ("src", "dst"):
            t = torch.randint(-2 ** 15, 2 ** 15, shape, device="cuda", generator=gen, dtype=torch.int32)
            s[name] = t if dt == torch.int32 else (t * 2.0 ** -12).to(dt)
        s["parent"] = torch.randint(0, W, (B, W), device="cuda", generator=gen, dtype=torch.int32)
        s["lengths"] = (torch.randint(1, case["T"] + 1, (B,), device="cuda", generator=gen,
                                      dtype=torch.int32) if case["ragged"] else None)
    return s


# ----------------------------------------------------------------------- run

def run(s):
    op, c = s["op"], s["case"]
    if own:
        lmh = _package()
        if op == "logits_lora":
            return lmh.lmhead_logits_lora(s["x"], s["W"], s["A"], s["B"], s["adapter"],
                                          scale=s["scale"], out_dtype=c["out"])
        if op == "lora_bwd":
            return lmh.lmhead_lora_bwd(s["g"], s["x"], s["A"], s["B"], s["adapter"], scale=s["scale"])
        if op == "beam_select":
            return lmh.lmhead_beam_select(s["logits"], s["scores"], n_out=c["out_beams"],
                                          finished=s["finished"], eos=s["eos"])
        return lmh.lmhead_beam_reorder(s["src"], s["parent"], out=s["dst"], beam_dim=1, len_dim=3,
                                       lengths=s["lengths"])
    if op == "logits_lora":
        return _plain_logits_lora(s)
    if op == "lora_bwd":
        return _plain_lora_bwd(s)
    if op == "beam_select":
        return _plain_beam_select(s)
    return _plain_beam_reorder(s)


def _own_columns(s):
    """[M, n r] FP32: the token's scale in the columns of its own adapter."""
    n, r, _ = s["A"].shape
    hot = (s["adapter"][:, None] == torch.arange(n, device="cuda")[None, :]).float()
    return (hot * s["scale"]).repeat_interleave(r, dim=1)


def _plain_logits_lora(s):
    A, B = s["A"].float(), s["B"].float()
    n, r, K = A.shape
    x = s["x"].float()
    u = (x @ A.reshape(n * r, K).t()) * _own_columns(s)
    z = x @ s["W"].float().t() + u @ B.permute(0, 2, 1).reshape(n * r, B.shape[1])
    return z.to(_TORCH[s["case"]["out"]])


def _plain_lora_bwd(s):
    A, B = s["A"].float(), s["B"].float()
    n, r, K = A.shape
    V = B.shape[1]
    x, g, own_cols = s["x"].float(), s["g"].float(), _own_columns(s)
    A2 = A.reshape(n * r, K)
    t = (g @ B.permute(1, 0, 2).reshape(V, n * r)) * own_cols
    u = (x @ A2.t()) * own_cols
    dX = t @ A2
    dA = (t.t() @ x).reshape(n, r, K)
    dB = (u.t() @ g).reshape(n, r, V).permute(0, 2, 1)
    return dX, dA, dB


def _plain_beam_select(s):
    # 64 bits: a rounding must not decide between two candidates
    B, W = s["scores"].shape
    z = s["logits"].double()
    V = z.shape[1]
    m = z.amax(1, keepdim=True)
    logz = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    c = (z - logz).reshape(B, W, V) + s["scores"].double()[:, :, None]
    c = torch.where(torch.isnan(c), torch.full_like(c, -math.inf), c)
    done = s["finished"]
    at_eos = (torch.arange(V, device="cuda") == s["eos"])[None, None, :]
    held = torch.where(at_eos, s["scores"].double()[:, :, None], torch.full_like(c, -math.inf))
    c = torch.where(done[:, :, None], held, c).reshape(B, W * V)
    k = s["case"]["out_beams"]
    best, at = torch.sort(c, dim=1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    parent, token = at // V, at % V
    ended = torch.gather(done, 1, parent) | (token == s["eos"])
    return best.float(), parent.to(torch.int32), token.to(torch.int32), ended


def _plain_beam_reorder(s):
    B, W = s["parent"].shape
    rows = (torch.arange(B, device="cuda")[:, None] * W + s["parent"]).reshape(-1)
    got = s["src"].index_select(1, rows)
    if s["lengths"] is None:
        return got
    T = s["src"].shape[3]
    live = torch.arange(T, device="cuda")[None, :] < s["lengths"].repeat_interleave(W)[:, None]
    return torch.where(live[None, :, None, :, None], got, s["dst"])


# ---------------------------------------------------------------- exact, work

def exact(case, seed):
    """The definition in 64 bits, adapter by adapter and request by request."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("logits_lora", "lora_bwd"):
        x, ids = s["x"].double(), s["adapter"].tolist()
        groups = {a: torch.tensor([m for m, q in enumerate(ids) if q == a], device="cuda")
                  for a in sorted(set(ids)) if a >= 0}
        A, B = s["A"].double(), s["B"].double()
        if op == "logits_lora":
            z = torch.matmul(x, s["W"].double().t())
            for a, rows in groups.items():
                u = torch.matmul(x[rows], A[a].t())
                z[rows] += float(s["scale"][a]) * torch.matmul(u, B[a].t())
            return z
        g = s["g"].double()
        dX, dA, dB = torch.zeros_like(x), torch.zeros_like(A), torch.zeros_like(B)
        for a, rows in groups.items():
            sc = float(s["scale"][a])
            t = torch.matmul(g[rows], B[a])
            dX[rows] = sc * torch.matmul(t, A[a])
            dA[a] = sc * torch.matmul(t.t(), x[rows])
            dB[a] = sc * torch.matmul(g[rows].t(), torch.matmul(x[rows], A[a].t()))
        return dX, dA, dB
    if op == "beam_select":
        B, W = s["scores"].shape
        V, k = case["V"], case["out_beams"]
        scores, parents, tokens, ended = [], [], [], []
        for b in range(B):
            cand = []
            for w in range(W):
                sc = float(s["scores"][b, w])
                if bool(s["finished"][b, w]):
                    cand.append((-sc, w, s["eos"]))
                    continue
                lp = torch.log_softmax(s["logits"][b * W + w].double(), 0) + sc
                kth = torch.topk(lp, min(k, V)).values[-1]
                idx = torch.nonzero(lp >= kth).flatten()
                cand += [(-v, w, i) for v, i in zip(lp[idx].tolist(), idx.tolist())]
            cand.sort()
            best = cand[:k]
            scores.append([-q[0] for q in best])
            parents.append([q[1] for q in best])
            tokens.append([q[2] for q in best])
            ended.append([q[2] == s["eos"] or bool(s["finished"][b, q[1]]) for q in best])
        return (torch.tensor(scores, dtype=torch.float64), torch.tensor(parents, dtype=torch.int32),
                torch.tensor(tokens, dtype=torch.int32), torch.tensor(ended))
    out = s["dst"].clone()
    W = case["W"]
    parents = s["parent"].tolist()
    for b in range(case["B"]):
        L = case["T"] if s["lengths"] is None else int(s["lengths"][b])
        for i in range(W):
            out[:, b * W + i, :, :L] = s["src"][:, b * W + parents[b][i], :, :L]
    return out


def work(case):
    op = case["op"]
    if op in ("logits_lora", "lora_bwd"):
        M, K, V, r = (case[k] for k in ("M", "K", "V", "r"))
        used = min(case["n"], M)
        adapters = used * r * (K + V) * 2
        if op == "logits_lora":
            out = 4 if case["out"] == "fp32" else 2
            return {"bytes": M * K * 2 + V * K * 2 + adapters + M * 4 + M * V * out,
                    "flops": 2.0 * M * K * V + 2.0 * M * r * (K + V)}
        return {"bytes": M * V * 2 + M * K * 2 + adapters + M * 4 + M * K * 4 + case["n"] * r * (K + V) * 4,
                "flops": 6.0 * M * r * (K + V)}
    if op == "beam_select":
        size = 4 if case["dtype"] == "fp32" else 2
        live = case["B"] * case["W"] * (1.0 - case["finished"])
        return {"bytes": live * case["V"] * size + case["B"] * (case["W"] * 5 + case["out_beams"] * 13),
                "flops": 4.0 * live * case["V"]}
    size = 2 if case["dtype"] == "bf16" else 4
    elems = case["layers"] * case["B"] * case["W"] * case["heads"] * case["T"] * case["D"]
    live = elems * (0.5 if case["ragged"] else 1.0)
    # a random parent map names 1 - (1 - 1/W)^W of the rows: those are read, all are written
    read = 1.0 - (1.0 - 1.0 / case["W"]) ** case["W"]
    return {"bytes": live * size * (1.0 + read), "flops": 0.0}
