"""Log-probabilities and distillation in 64 bits over the whole vocabulary, and
the error bounds of the kernels' arithmetic, for the GPU tests.

Bounds (u = 2^-24, half a step of FP32, as every other rounding's relative
size): the kernels form y = (z - m) c with c = log2(e) (1 / T), so y is off by
at most 5 u |y| (difference, quotient, constant, two products) and exp2 by 2 u;
a term's exponential is off by (5 |x| + 2) u of itself, x = y ln 2.  Of the sum
d, weighted by p, that is 5 u E|x| + 2 u, and E|x| = H - log d' <= ln V (d' >= 1);
a further exponential where waves meet (2 u), at
most 31 + 6 additions of a lane's segment and of a wave in FP32 (37 u, the rest is
FP64) and the rounding of d itself.  A lane takes up to V / 8192 segments (four waves
of 2048 columns); each further one multiplies the sum so far by an exponential and
adds to it (4 u).  d is therefore within (5 ln V + 42 + 4 V / 8192) u of itself, and
log d within as much absolutely.  (The one-read kernel adds 15 + 2 + 6 times.)"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -120  # what FP32 may lose below its range


def d_bound(V):
    return (5.0 * math.log(max(V, 2)) + 42.0 + 4.0 * (V // 8192)) * U


def temperatures(temperature, n, device):
    if temperature is None:
        return torch.ones(n, 1, dtype=torch.float64, device=device)
    return temperature.double().expand(n).reshape(n, 1)


def log_softmax(z, T):
    """(x, log p, m, d) in 64 bits; columns at -inf give x = log p = -inf."""
    z = z.double()
    m = z.amax(1, keepdim=True)
    x = (z - m) / T
    d = torch.exp(x).sum(1, keepdim=True)
    return x, x - torch.log(d), m, d


def logprobs(z, token, temperature, ignore=-100):
    """dict of logprob, entropy, rank, m, d and the tolerances of the first two;
    rows are assumed to be finite somewhere and free of NaN and +inf."""
    n, V = z.shape
    T = temperatures(temperature, n, z.device)
    x, lp, m, d = log_softmax(z, T)
    p = torch.exp(lp)
    zero = torch.zeros_like(p)
    ax = torch.where(p > 0, x.abs(), zero)
    entropy = -torch.where(p > 0, p * lp, zero).sum(1)
    ex, ex2 = (p * ax).sum(1), (p * ax * ax).sum(1)
    rel = d_bound(V)
    out = {"entropy": entropy, "m": m[:, 0], "d": d[:, 0], "p": p, "lp": lp, "x": ax,
           "tol_d": rel * d[:, 0] + TINY,
           # s / d: each term's exponential, y and product; its sum; d
           "tol_entropy": rel * (1.0 + ex) + 5 * U * ex2 + 52 * U * ex + U * entropy.abs() + TINY, "T": T}
    if token is not None:
        y = token.long()
        ok = (y >= 0) & (y < V)
        at = y.clamp(0, V - 1)[:, None]
        got = torch.gather(lp, 1, at)[:, 0]
        zy = torch.gather(z.double(), 1, at)
        ahead = (z.double() > zy) | ((z.double() == zy) & (torch.arange(V, device=z.device)[None] < at))
        nan = torch.full_like(got, math.nan)
        out["logprob"] = torch.where(y == ignore, torch.zeros_like(got), torch.where(ok, got, nan))
        out["rank"] = torch.where((y == ignore) | ~ok, -1, ahead.sum(1)).to(torch.int32)
        finite = torch.where(torch.isinf(got), torch.zeros_like(got), got)
        out["tol_logprob"] = rel + 4 * U * finite.abs()
    return out


def top(z, k):
    """(columns, values) of the k largest, equal ones by ascending column; -1
    and -inf where fewer lie above -inf."""
    v, i = torch.sort(z.double() + 0.0, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    return torch.where(v > -math.inf, i, -1), v


def logprobs_grad(z, token, temperature, g, h, ignore=-100):
    """(gradient, tolerance in FP32) of sum g log p_y + h H."""
    n, V = z.shape
    r = logprobs(z, None, temperature)
    p, T, x = r["p"], r["T"], r["x"]
    lp = torch.where(p > 0, r["lp"], torch.zeros_like(p))
    H = r["entropy"][:, None]
    g = torch.zeros(n, 1, dtype=torch.float64, device=z.device) if g is None else g.double().expand(n)[:, None]
    h = torch.zeros(n, 1, dtype=torch.float64, device=z.device) if h is None else h.double().expand(n)[:, None]
    if token is None:
        g = torch.zeros_like(g)
        hot = torch.zeros_like(p)
    else:
        y = token.long()[:, None]
        g = torch.where(y == ignore, torch.zeros_like(g), g)
        hot = torch.zeros_like(p).scatter_(1, y.clamp(min=0), 1.0) * (y != ignore)
    out = (g * (hot - p) - h * p * (lp + H)) / T
    rel = d_bound(V)
    part = rel + (5 * x + 12) * U
    log_d = torch.log(r["d"])[:, None]
    tol = p * g.abs() * part + p * h.abs() * ((lp.abs() + H.abs()) * part + r["tol_entropy"][:, None] + 2 * rel +
                                              8 * U * (x + log_d + H.abs()))
    tol = (tol + hot * g.abs() * 4 * U) / T + TINY
    bad = (g == 0) & (h == 0)
    return torch.where(bad, torch.zeros_like(out), out), tol


def distill(z, ids, values, tail, temperature, dloss):
    """dict of loss, dlogits and their tolerances (the gradient's in FP32)."""
    n, V = z.shape
    T = temperatures(temperature, n, z.device)
    x, lp, m, d = log_softmax(z, T)
    ids, values = ids.long(), values.double()
    there = (ids >= 0) & (values > -math.inf)
    held = there.any(1)
    k = ids.shape[1]
    vt = values if tail else values / T
    if k and not tail:
        vt = vt - torch.where(held[:, None], torch.logsumexp(torch.where(there, vt, -math.inf), 1, keepdim=True),
                              torch.zeros_like(T))
    zero = torch.zeros(n, max(k, 1), dtype=torch.float64, device=z.device)[:, :k]
    q = torch.where(there, torch.exp(vt), zero)
    at = ids.clamp(min=0)
    lp_at = torch.gather(lp, 1, at)
    loss = torch.where(q > 0, q * (torch.where(q > 0, vt, zero) - lp_at), zero).sum(1)
    xt = torch.where(there, vt.abs(), zero)
    most = xt.amax(1) if k else torch.zeros(n, dtype=torch.float64, device=z.device)
    rel = d_bound(V)
    fin = torch.where(q > 0, lp_at.abs(), zero)
    fin = torch.where(torch.isinf(fin), zero, fin)
    # 1 / T rounded moves every x_l by u |x_l|, so log q by 2 u max |x|
    tol_loss = (q * (rel + 5 * U * fin + 4 * U * most[:, None]) + q * 4 * U * most[:, None] * (fin + xt)).sum(1)
    weight = q.sum(1)
    p = torch.exp(lp)
    taken = torch.zeros(n, V + 1, dtype=torch.bool, device=z.device)
    taken.scatter_(1, torch.where(there, ids, V), True)
    taken = taken[:, :V]
    qv = torch.zeros(n, V + 1, dtype=torch.float64, device=z.device)
    qv.scatter_add_(1, torch.where(there, ids, V), q)
    qv = qv[:, :V]
    off = weight[:, None] * p
    mag = off
    if tail:
        rest = torch.where(taken, torch.full_like(lp, -math.inf), lp)
        log_r = torch.logsumexp(rest, 1)
        some = log_r > -math.inf
        q_r = torch.where(some, (1.0 - weight).clamp(min=0.0), torch.zeros_like(weight))
        has = q_r > 0
        loss = loss + torch.where(has, q_r * (torch.log(q_r) - log_r), torch.zeros_like(loss))
        tol_loss = tol_loss + torch.where(has, q_r * (2 * rel + 5 * U * log_r.abs()), torch.zeros_like(loss))
        weight = weight + q_r
        cond = torch.exp(torch.where(taken | ~some[:, None], torch.full_like(lp, -math.inf), lp - log_r[:, None]))
        off = weight[:, None] * p - q_r[:, None] * cond
        mag = weight[:, None] * p + q_r[:, None] * cond
    ax = torch.where(x > -math.inf, x.abs(), torch.zeros_like(x))
    ax = torch.where(p > 0, ax, torch.zeros_like(ax))
    grad = torch.where(taken, weight[:, None] * p - qv, off)
    tol = mag * (2 * rel + (10 * ax + 16) * U) + qv * (5 * most[:, None] + 16) * 2 * U
    up = dloss.double().expand(n)[:, None] / T
    live = held[:, None] & (up != 0)
    return {"loss": torch.where(held, loss, torch.zeros_like(loss)),
            "tol_loss": tol_loss + 2 * U * loss.abs() + TINY,
            "dlogits": torch.where(live, grad * up, torch.zeros_like(grad)),
            "tol_dlogits": tol * up.abs() + 4 * U * (grad * up).abs() + TINY, "weight": weight, "m": m[:, 0],
            "d": d[:, 0]}


def assert_within(got, want, tol, what):
    """|got - want| <= tol plus got's own rounding; infinities and NaN equal."""
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: {got[i].item()!r} for "
                             f"{want[i].item()!r}, tolerance {(tol.expand_as(want))[i].item()!r}")


def assert_grad(got, want, tol, what):
    assert_within(got, want, tol + (HALF[got.dtype] * want.abs() * 1.01 if got.dtype != torch.float32 else U * want.abs()),
                  what)


def padded(n, V, dtype, fill=math.nan, extra=8):
    """[n, V] in a buffer of wider rows that holds `fill`."""
    mult = 8 if dtype == torch.bfloat16 else 4
    ld = (V + mult - 1) // mult * mult + extra
    return torch.full((n, ld), fill, dtype=dtype, device="cuda")[:, :V]


def repad(t):
    """A copy in a padded buffer."""
    out = padded(*t.shape, t.dtype)
    out.copy_(t)
    return out


def padding_holds(t):
    base = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
    return bool(torch.isnan(base[:, t.shape[1]:].float()).all())


def random_logits(n, V, dtype, seed, sigma=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = padded(n, V, dtype)
    z.copy_(sigma * torch.randn(n, V, device="cuda", generator=gen))
    return z, gen
