"""Adapter logits and adapter gradients against plain 64-bit formulas.

Integer operands with sums below 2^24 make every product and sum exact in
FP32 whatever its order, so those cases are compared bit for bit.  For random
operands the bound is the FP32 accumulation's: a product over n terms in 16-
or 32-deep matrix steps adds at most n / 16 partial sums one after another,
plus a fixed number of joins (waves, pieces, parts), each off by at most 2^-24
of the sum of absolute products."""
import numpy as np
import pytest
import torch

import lm_head_fp32_amd as lmh

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


def _say(*a):
    print(*a, flush=True)


def _padded(t, pad):
    """The same values as a view whose rows are `pad` elements further apart
    (rounded up to 16 bytes), NaN in between."""
    mult = 16 // t.element_size()
    ld = (t.shape[-1] + pad + mult - 1) // mult * mult
    buf = torch.full((*t.shape[:-1], ld), float("nan"), dtype=t.dtype, device=t.device)
    buf[..., : t.shape[-1]] = t
    return buf[..., : t.shape[-1]]


def _untouched(view):
    base = view.as_strided((*view.shape[:-1], view.stride(-2)), view.stride())
    return bool(torch.isnan(base[..., view.shape[-1]:]).all())


def _ints(g, shape, hi, dtype=torch.bfloat16):
    return torch.randint(-hi, hi + 1, shape, device="cuda", generator=g).to(dtype)


def _ids(g, M, n, order, invalid=False):
    if n == 0:
        ids = torch.full((M,), -1, device="cuda")
    else:
        ids = torch.randint(0, n, (M,), device="cuda", generator=g)
    if order == "runs":
        ids = ids.sort().values
    ids[torch.rand(M, device="cuda", generator=g) < 0.1] = -1
    if invalid and M > 2:
        ids[1] = n
        ids[M // 2] = 2 ** 31 - 1
        ids[M - 1] = -(2 ** 31)
    return ids.to(torch.int32)


def _case(M, K, V, r, n, order, seed, pad, invalid=False, hi=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, W = _padded(_ints(g, (M, K), hi), pad), _padded(_ints(g, (V, K), hi), pad)
    A, B = _padded(_ints(g, (n, r, K), 1), pad), _padded(_ints(g, (n, V, r), hi), pad)
    scale = torch.tensor([1.0, 2.0, 0.5, -1.0], device="cuda")[torch.arange(n, device="cuda") % 4]
    return x, W, A, B, _ids(g, M, n, order, invalid), scale, g


def _ref_logits(x, W, A, B, ids, scale):
    """(logits, sum of absolute products) in 64 bits."""
    xd = x.double()
    z, S = xd @ W.double().t(), xd.abs() @ W.double().abs().t()
    for a in range(A.shape[0]):
        rows = (ids == a).nonzero().flatten()
        if rows.numel():
            s = 1.0 if scale is None else scale[a].double()
            z[rows] += s * ((xd[rows] @ A[a].double().t()) @ B[a].double().t())
            S[rows] += abs(s) * ((xd[rows].abs() @ A[a].double().abs().t()) @ B[a].double().abs().t())
    z[ids >= A.shape[0]] = float("nan")
    return z, S


# M, K, V, rank, adapters: one token, odd sizes, ranks at and between the
# kernels' 16 / 32 / 64 / 128, more adapters than tokens, each kernel of the
# shared product (few tokens, ring, large tiles, whole tiles).
SHAPES = [(1, 512, 1000, 16, 3), (3, 40, 257, 1, 2), (16, 24, 31, 7, 16), (17, 128, 33, 5, 4),
          (64, 264, 515, 8, 1), (100, 520, 1001, 12, 7), (130, 1032, 700, 24, 40),
          (257, 96, 300, 64, 5), (300, 72, 260, 128, 3), (33, 8200, 260, 100, 50),
          (700, 4104, 520, 33, 9), (1024, 128, 32768, 16, 4)]


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("M,K,V,r,n", SHAPES)
def test_logits_integers_exact(M, K, V, r, n, order, out):
    _say("lora logits", M, K, V, r, n, order, out)
    # the largest sum: K 9 + r (K 3) 3 2 stays below 2^24 for typical sums
    x, W, A, B, ids, scale, _ = _case(M, K, V, r, n, order, 7 + M + r, 8, invalid=True)
    z, S = _ref_logits(x, W, A, B, ids, scale)
    dt = torch.float32 if out == "fp32" else torch.bfloat16
    dst = _padded(torch.full((M, V), float("nan"), dtype=dt, device="cuda"), 8)
    assert lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out=dst) is dst
    torch.cuda.synchronize()
    exact = bool((S < 2 ** 24).all())
    want = z.float() if out == "fp32" else z.float().to(torch.bfloat16)
    if exact:
        assert torch.equal(torch.nan_to_num(dst, nan=1e30), torch.nan_to_num(want, nan=1e30))
    else:
        tol = (K / 16 + 64) * EPS * S + (z.abs() * 2.0 ** -8 if out == "bf16" else 0.0)
        ok = ~torch.isnan(z)
        assert torch.equal(torch.isnan(dst), ~ok)
        assert ((dst.double() - z).abs()[ok] <= tol[ok]).all()
    assert _untouched(dst)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,n,r", [(257, 1, 16), (1023, 40, 20), (1025, 200, 16), (2100, 3, 70), (5000, 700, 3)])
def test_logits_of_large_mixed_batches(M, n, r, out):
    """Batches beyond one window of the tokens' order, none of it in runs."""
    test_logits_integers_exact(M, 64, 270, r, n, "mixed", out)


def test_logits_of_large_batches_without_adapters():
    x, W, A, B, ids, scale, _ = _case(300, 64, 270, 8, 0, "mixed", 3, 0)
    ids[7], ids[299] = 0, 5  # no adapters, so none with these numbers
    want = x.double() @ W.double().t()
    want[7] = want[299] = float("nan")
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty((300, 272), dtype=dt, device="cuda")[:, :270]
        lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out=out)
        assert torch.equal(torch.nan_to_num(out, nan=1e30), torch.nan_to_num(want.float().to(dt), nan=1e30))


@pytest.mark.parametrize("M,K,V,r,n", [(1, 4096, 2000, 16, 8), (37, 2040, 3003, 12, 5),
                                       (128, 1024, 2048, 64, 32), (513, 2048, 1025, 128, 4)])
def test_logits_random(M, K, V, r, n):
    _say("lora logits random", M, K, V, r, n)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    W = _padded((0.02 * torch.randn(V, K, device="cuda", generator=g)).bfloat16(), 0)
    A = (K ** -0.5 * torch.randn(n, r, K, device="cuda", generator=g)).bfloat16()
    B = _padded(torch.randn(n, V, r, device="cuda", generator=g).bfloat16(), 0)
    scale = torch.rand(n, device="cuda", generator=g) * 4
    ids = _ids(g, M, n, "mixed")
    z, S = _ref_logits(x, W, A, B, ids, scale)
    got = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out_dtype="fp32")
    b16 = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale)
    torch.cuda.synchronize()
    # K / 16 sequential sums, 16 wave parts, 3 r / 16 piece steps, the scale
    tol = (K / 16 + 16 + 3 * 128 / 16 + 4) * EPS * S
    assert ((got.double() - z).abs() <= tol).all()
    assert torch.equal(b16, got.to(torch.bfloat16))  # one rounding of the same FP32 sum


def test_no_adapter_is_the_plain_product():
    g = torch.Generator(device="cuda").manual_seed(3)
    x, W, A, B, _, scale, _ = _case(40, 96, 130, 8, 2, "mixed", 3, 0)
    none = torch.full((40,), -5, dtype=torch.int32, device="cuda")
    for dt in ("fp32", "bf16"):
        want = lmh.lmhead_logits(x, W, out_dtype=dt)
        assert torch.equal(lmh.lmhead_logits_lora(x, W, A, B, none, out_dtype=dt), want)
        # no adapter loaded at all
        assert torch.equal(lmh.lmhead_logits_lora(x, W, A[:0], B[:0], none, out_dtype=dt), want)
    # scale None is 1; an empty contraction and an empty batch
    ids = torch.zeros(40, dtype=torch.int32, device="cuda")
    one = torch.ones(2, device="cuda")
    assert torch.equal(lmh.lmhead_logits_lora(x, W, A, B, ids, out_dtype="fp32"),
                       lmh.lmhead_logits_lora(x, W, A, B, ids, scale=one, out_dtype="fp32"))
    z = lmh.lmhead_logits_lora(x[:, :0], W[:, :0], A[:, :, :0], B, ids, out_dtype="fp32")
    assert z.shape == (40, 130) and not z.any()
    assert lmh.lmhead_logits_lora(x[:0], W, A, B, ids[:0], out_dtype="fp32").shape == (0, 130)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("M", [20, 300])
def test_requests_do_not_touch_each_other(M, value):
    """A non-finite weight of one adapter, and a non-finite token, stay in their
    own rows, in the logits and in the gradients."""
    x, W, A, B, ids, scale, g = _case(M, 136, 140, 12, 4, "mixed", 11, 8)
    ids[0], ids[1] = 2, 1
    gr = _ints(g, (M, 140), 2)
    gr = _padded(gr, 0)
    clean = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out_dtype="fp32")
    cdX, cdA, cdB = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale)
    A2, B2 = A.clone(), B.clone()
    A2[2, 3, 5] = value
    B2[2, 7, 1] = value
    A2, B2 = _padded(A2, 8), _padded(B2, 8)
    got = lmh.lmhead_logits_lora(x, W, A2, B2, ids, scale=scale, out_dtype="fp32")
    dX, dA, dB = lmh.lmhead_lora_bwd(gr, x, A2, B2, ids, scale=scale)
    other = ids != 2
    assert torch.equal(got[other], clean[other]) and not torch.isfinite(got[~other]).all()
    assert torch.equal(dX[other], cdX[other])
    keep = [0, 1, 3]
    assert torch.equal(dA[keep], cdA[keep]) and torch.equal(dB[keep], cdB[keep])
    x2 = x.clone()
    x2[0, 4] = value
    g2 = gr.clone()
    g2[0, 4] = value
    x2, g2 = _padded(x2, 0), _padded(g2, 0)
    got = lmh.lmhead_logits_lora(x2, W, A, B, ids, scale=scale, out_dtype="fp32")
    assert torch.equal(got[1:], clean[1:])
    dX, dA, dB = lmh.lmhead_lora_bwd(g2, x2, A, B, ids, scale=scale)
    assert torch.equal(dX[1:], cdX[1:])
    assert torch.equal(dA[keep], cdA[keep]) and torch.equal(dB[keep], cdB[keep])
    assert not torch.isfinite(dX[0]).all()


def _ref_bwd(gr, x, A, B, ids, scale):
    xd, gd = x.double(), gr.double()
    dX, dA, dB = torch.zeros_like(xd), torch.zeros_like(A, dtype=torch.float64), torch.zeros_like(
        B, dtype=torch.float64)
    SX, SA, SB = torch.zeros_like(dX), torch.zeros_like(dA), torch.zeros_like(dB)
    for a in range(A.shape[0]):
        rows = (ids == a).nonzero().flatten()
        if not rows.numel():
            continue
        s, Aa, Ba = (1.0 if scale is None else scale[a].double()), A[a].double(), B[a].double()
        t, u = s * (gd[rows] @ Ba), s * (xd[rows] @ Aa.t())
        ta = abs(s) * (gd[rows].abs() @ Ba.abs())
        ua = abs(s) * (xd[rows].abs() @ Aa.abs().t())
        dX[rows], dA[a], dB[a] = t @ Aa, t.t() @ xd[rows], gd[rows].t() @ u
        SX[rows], SA[a], SB[a] = ta @ Aa.abs(), ta.t() @ xd[rows].abs(), gd[rows].abs().t() @ ua
    dX[ids >= A.shape[0]] = float("nan")
    return (dX, dA, dB), (SX, SA, SB)


@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("M,K,V,r,n", SHAPES[:-1] + [(1024, 520, 2056, 16, 4), (70, 300, 270, 4, 130)])
def test_bwd_integers_exact(M, K, V, r, n, order):
    _say("lora bwd", M, K, V, r, n, order)
    K8 = (K + 7) // 8 * 8
    x, W, A, B, ids, scale, g = _case(M, K8, V, r, n, order, 50 + M + r, 8, invalid=True, hi=1)
    gr = _padded(_ints(g, (M, V), 1), 8)
    want, sums = _ref_bwd(gr, x, A, B, ids, scale)
    outs = (_padded(torch.full((M, K8), float("nan"), device="cuda"), 4),
            _padded(torch.full((n, r, K8), float("nan"), device="cuda"), 4),
            _padded(torch.full((n, V, r), float("nan"), device="cuda"), 4))
    got = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale, dX=outs[0], dA=outs[1], dB=outs[2])
    torch.cuda.synchronize()
    for o, q, w, S, name in zip(outs, got, want, sums, ("dX", "dA", "dB")):
        assert q is o and _untouched(o), name
        assert (S < 2 ** 24).all(), name  # so every sum is exact
        assert torch.equal(torch.nan_to_num(o, nan=1e30), torch.nan_to_num(w.float(), nan=1e30)), name
    # each output alone, the others skipped, and adding to what is there
    for i, name in enumerate(("dX", "dA", "dB")):
        one = [False, False, False]
        one[i] = torch.full_like(outs[i], 3.0)
        one[i] = _padded(one[i], 4)
        kw = dict(zip(("dX", "dA", "dB"), one))
        res = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale, accumulate=True, **kw)
        assert [t is None for t in res] == [j != i for j in range(3)]
        assert torch.equal(torch.nan_to_num(one[i], nan=1e30),
                           torch.nan_to_num(want[i].float() + 3.0, nan=1e30)), name
        assert _untouched(one[i])


@pytest.mark.parametrize("M,n", [(90, 1022), (90, 1023), (400, 1022), (400, 1200)])
def test_bwd_many_adapters(M, n):
    """More adapters than are grouped beside the first product, and just as many."""
    test_bwd_integers_exact(M, 40, 30, 2, n, "mixed")


@pytest.mark.parametrize("M,K,V,r,n", [(101, 2048, 3003, 8, 3), (256, 1024, 2048, 64, 2),
                                       (40, 512, 1000, 128, 2)])
def test_bwd_random(M, K, V, r, n):
    _say("lora bwd random", M, K, V, r, n)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    A = (K ** -0.5 * torch.randn(n, r, K, device="cuda", generator=g)).bfloat16()
    B = _padded((0.1 * torch.randn(n, V, r, device="cuda", generator=g)).bfloat16(), 0)
    gr = _padded((1e-3 * torch.randn(M, V, device="cuda", generator=g)).bfloat16(), 0)
    scale = torch.rand(n, device="cuda", generator=g) * 4
    ids = _ids(g, M, n, "mixed")
    want, sums = _ref_bwd(gr, x, A, B, ids, scale)
    got = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale)
    torch.cuda.synchronize()
    # the inner sum over K or V in 32-deep steps and its joins (16 waves, or
    # ceil(V / 256) parts), the outer over r or M, three pieces each, the scale
    inner = max(K / 32 + 16, 8 + V / 256) + 4
    for q, w, S, steps, name in zip(got, want, sums, (3 * 128 / 32, 3 * M / 32 + 3, 3 * M / 32 + 3),
                                    ("dX", "dA", "dB")):
        tol = (inner + steps + 4) * EPS * S
        assert ((q.double() - w).abs() <= tol).all(), name
    again = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale)
    for q, p in zip(got, again):
        assert torch.equal(q, p)


@pytest.mark.parametrize("M,K,V,r,n", [
    (12, 7976, 1000, 4, 3), (16, 8192, 1000, 4, 3), (45, 5112, 2601, 8, 5), (45, 5120, 2601, 8, 5),
    (100, 1000, 4000, 16, 2), (200, 520, 3001, 8, 4), (257, 264, 5000, 8, 4), (900, 4632, 1001, 4, 3)])
def test_logits_of_few_tiles(M, K, V, r, n):
    """Outputs that one workgroup per tile and all of K would leave most CUs out of."""
    for out in ("fp32", "bf16"):
        test_logits_integers_exact(M, K, V, r, n, "mixed", out)


@pytest.mark.parametrize("M,K,V,r,n", [(1, 1, 1, 1, 1), (5, 1, 9, 3, 2), (2, 7, 3, 2, 1), (300, 3, 5, 128, 2),
                                       (70001, 32, 40, 4, 3)])
def test_smallest_and_longest_batches(M, K, V, r, n):
    test_logits_integers_exact(M, K, V, r, n, "mixed", "fp32")
    test_logits_integers_exact(M, K, V, r, n, "runs", "bf16")
    test_bwd_integers_exact(M, K, V, r, n, "mixed")


def test_offsets_past_32_bits():
    """Logits and gradients of more than 2^31 elements: the last tokens' results
    are those of a call that holds them alone."""
    M, K, V, r, n, last = 66000, 64, 32800, 4, 2, 40
    x, W, A, B, ids, scale, g = _case(M, K, V, r, n, "mixed", 11, 0)
    ids[:M - last] = -1  # they alone have adapters
    rows = slice(M - last, M)
    tail = _padded(x[rows].clone(), 0), ids[rows].clone()
    for dt in ("fp32", "bf16"):
        z = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out_dtype=dt)
        # integers of at most 9 K + 18 r K, far below 2^24, so every sum is exact
        assert torch.equal(z[rows], lmh.lmhead_logits_lora(tail[0], W, A, B, tail[1], scale=scale, out_dtype=dt))
        del z
    gr = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    gr[rows] = _ints(g, (last, V), 1)
    got = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale)
    want = lmh.lmhead_lora_bwd(gr[rows].clone(), tail[0], A, B, tail[1], scale=scale)
    assert torch.equal(got[0][rows], want[0]) and not got[0][:M - last].any()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_bwd_empty_sizes():
    x, W, A, B, ids, scale, g = _case(20, 64, 72, 8, 3, "mixed", 5, 0)
    gr = _ints(g, (20, 72), 1)
    # no tokens: zeros in dA and dB, or what was there when adding
    dX, dA, dB = lmh.lmhead_lora_bwd(gr[:0], x[:0], A, B, ids[:0])
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()
    dA.fill_(2.0)
    lmh.lmhead_lora_bwd(gr[:0], x[:0], A, B, ids[:0], dX=False, dA=dA, dB=False, accumulate=True)
    assert (dA == 2.0).all()
    # no adapters: zeros in dX
    none = torch.full_like(ids, -1)
    dX, dA, dB = lmh.lmhead_lora_bwd(gr, x, A[:0], B[:0], none)
    assert not dX.any() and dA.shape == (0, 8, 64) and dB.shape == (0, 72, 8)
    # an empty vocabulary: zeros everywhere
    dX, dA, dB = lmh.lmhead_lora_bwd(gr[:, :0], x, A, B[:, :0], ids)
    assert not dX.any() and not dA.any() and dB.shape == (3, 0, 8)


def test_gradients_are_the_differences():
    """The loss sum(g z) is linear in each of x (the adapters' part), A and B:
    with integers its difference for a unit step is the gradient exactly."""
    M, K, V, r, n = 33, 48, 70, 6, 3
    x, W, A, B, ids, _, g = _case(M, K, V, r, n, "mixed", 21, 0, hi=2)
    scale = torch.tensor([1.0, 2.0, -1.0], device="cuda")
    gr = _padded(_ints(g, (M, V), 2), 0)
    W0 = torch.zeros_like(W)

    def loss(x_, A_, B_):
        z = lmh.lmhead_logits_lora(x_, W0, A_, B_, ids, scale=scale, out_dtype="fp32")
        return float((z.double() * gr.double()).sum())

    dX, dA, dB = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale)
    base = loss(x, A, B)
    rng = np.random.default_rng(1)
    for t, grad, which in ((x, dX, 0), (A, dA, 1), (B, dB, 2)):
        for _ in range(6):
            at = tuple(int(rng.integers(0, d)) for d in t.shape)
            t2 = _padded(t.clone(), 0)
            t2[at] += 1
            args = [x, A, B]
            args[which] = t2
            assert loss(*args) - base == float(grad[at]), (which, at)


def test_training_step_with_adapters():
    """Adapter logits, their cross-entropy and BF16 gradient, and the whole
    input gradient: the shared part from lmhead_dgrad, the adapters' added."""
    M, K, V, r, n = 130, 256, 1000, 8, 3
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    W = (0.05 * torch.randn(V, K, device="cuda", generator=g)).bfloat16()
    A = (K ** -0.5 * torch.randn(n, r, K, device="cuda", generator=g)).bfloat16()
    B = (0.2 * torch.randn(n, V, r, device="cuda", generator=g)).bfloat16()
    scale = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    ids = _ids(g, M, n, "mixed")
    target = torch.randint(0, V, (M,), device="cuda", generator=g, dtype=torch.int32)
    target[::9] = -100
    z = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out_dtype="fp32")
    _, inv = lmh.lmhead_xent_mean(None, target)
    loss, _, gr = lmh.lmhead_xent_fused(z, target, inv, grad_dtype="bf16")
    dX = lmh.lmhead_dgrad(gr, W, dx_dtype="fp32")
    dA, dB = torch.zeros(n, r, K, device="cuda"), torch.zeros(n, V, r, device="cuda")
    lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale, dX=dX, dA=dA, dB=dB, accumulate=True)
    torch.cuda.synchronize()
    # loss from the 64-bit logits: z is off by at most the accumulation bound
    zd, S = _ref_logits(x, W, A, B, ids, scale)
    lz = torch.logsumexp(zd, 1)
    valid = target >= 0
    want = lz - zd.gather(1, target.clamp(min=0).long()[:, None])[:, 0]
    tol = 2 * (K / 16 + 64) * EPS * S.amax(1) + 1e-5 * want.abs().clamp(min=1)
    assert ((loss.double() - want).abs()[valid] <= tol[valid]).all()
    (rX, rA, rB), (SX, SA, SB) = _ref_bwd(gr, x, A, B, ids, scale)
    rX += gr.double() @ W.double()
    SX += gr.double().abs() @ W.double().abs()
    for q, w, s in ((dX, rX, SX), (dA, rA, SA), (dB, rB, SB)):
        assert ((q.double() - w).abs() <= (V / 16 + 128) * EPS * s).all()


def test_streams_workspaces_and_graphs():
    """The calls on a stream of their own, two at once with a workspace each,
    and captured: replays match the eager result bitwise."""
    M, K, V, r, n = 48, 520, 1000, 16, 5
    x, W, A, B, ids, scale, g = _case(M, K, V, r, n, "mixed", 31, 0)
    x2 = _ints(g, (M, K), 3)
    gr = _ints(g, (M, V), 1)
    want = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out_dtype="bf16")
    want2 = lmh.lmhead_logits_lora(x2, W, A, B, ids, scale=scale, out_dtype="fp32")
    back = lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    out1, out2 = torch.empty_like(want), torch.empty_like(want2)
    for _ in range(4):
        lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out=out1, stream=s1)
        lmh.lmhead_logits_lora(x2, W, A, B, ids, scale=scale, out=out2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(out1, want) and torch.equal(out2, want2)
    with pytest.raises(ValueError):  # a raw handle needs the caller's workspace
        lmh.lmhead_logits_lora(x, W, A, B, ids, out=out1, stream=s1.cuda_stream)
    ws = torch.empty(max(lmh.lmhead_logits_lora_workspace_bytes(M, K, V, r, "bf16"),
                         lmh.lmhead_lora_bwd_workspace_bytes(M, K, V, r, n)), dtype=torch.uint8,
                     device="cuda")
    outs = [torch.empty_like(want)] + [torch.empty_like(t) for t in back]

    def step():
        lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out=outs[0], workspace=ws)
        lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale, dX=outs[1], dA=outs[2], dB=outs[3],
                            workspace=ws)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs over one workspace, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
    for rep in range(4):
        for t in outs:
            t.zero_()
        ws.fill_(0xff)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, (want, *back)):
            assert torch.equal(t, w), rep
        step()
        torch.cuda.synchronize()
    # the ids are read at replay: another batch needs no new capture
    ids.copy_(torch.full_like(ids, 1))
    fresh = lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out_dtype="bf16")
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fresh)


@pytest.mark.parametrize("M,V,out", [(600, 1000, "fp32"), (600, 20000, "fp32"), (1500, 3000, "bf16"), (40, 20000, "bf16")])
def test_captured_batches_of_other_adapters(M, V, out):
    """A captured step replayed with other ids in place, over a workspace of NaNs."""
    K, r, n = 136, 16, 7
    x, W, A, B, ids, scale, g = _case(M, K, V, r, n, "mixed", 41, 0)
    gr = _ints(g, (M, V), 1)
    if V % 8:
        gr = _padded(gr, 0)
    ws = torch.empty(max(lmh.lmhead_logits_lora_workspace_bytes(M, K, V, r, out),
                         lmh.lmhead_lora_bwd_workspace_bytes(M, K, V, r, n)), dtype=torch.uint8, device="cuda")
    z = torch.empty((M, V), dtype=torch.float32 if out == "fp32" else torch.bfloat16, device="cuda")
    grads = [torch.empty(t.shape, device="cuda") for t in (x, A, B)]

    def step():
        lmh.lmhead_logits_lora(x, W, A, B, ids, scale=scale, out=z, workspace=ws)
        lmh.lmhead_lora_bwd(gr, x, A, B, ids, scale=scale, dX=grads[0], dA=grads[1], dB=grads[2], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(4):
        ids.copy_(_ids(g, M, n, "runs" if rep % 2 else "mixed", invalid=rep == 2))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (z, *grads)]
        for t in (z, *grads):
            t.fill_(7.0)
        ws.fill_(0xff)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((z, *grads), want):
            assert torch.equal(torch.nan_to_num(t, nan=1e30), torch.nan_to_num(w, nan=1e30)), rep
