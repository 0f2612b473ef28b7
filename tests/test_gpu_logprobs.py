"""Log-probabilities of given tokens, entropies, ranks, alternatives and their
gradient, against the definitions in 64 bits (tests/row_reference.py)."""
import math

import pytest
import torch

import lm_head_fp32_amd as lmh
import row_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


def _temperature(kind, n, gen):
    if kind == "none":
        return None
    t = 0.5 + torch.rand(1 if kind == "one" else n, device="cuda", generator=gen)
    return t


def _tokens(n, V, gen):
    t = torch.randint(0, V, (n,), device="cuda", generator=gen)
    return torch.where(torch.arange(n, device="cuda") % 5 == 3, -100, t).to(torch.int32)


def _check_forward(z, token, temperature, k, got=None):
    n, V = z.shape
    got = got or lmh.lmhead_logprobs(z, token, temperature=temperature, n_top=k)
    lp, ent, rank, top_lp, top_tok, stats = got
    want = ref.logprobs(z, token, temperature)
    ref.assert_within(ent, want["entropy"], want["tol_entropy"], "entropy")
    ref.assert_within(stats[:, 0], want["m"], 0 * want["m"], "m")
    ref.assert_within(stats[:, 1], want["d"], want["tol_d"], "d")
    assert torch.equal(stats[:, 2], ent)
    if token is None:
        assert lp is None and rank is None
        assert (stats[:, 3] == 0).all()
    else:
        ref.assert_within(lp, want["logprob"], want["tol_logprob"], "logprob")
        assert torch.equal(rank, want["rank"])
        assert torch.equal(stats[:, 3].nan_to_num(7.0), lp.nan_to_num(7.0))
    if k:
        idx, val = ref.top(z, k)
        assert torch.equal(top_tok.long(), idx)
        there = torch.where(idx >= 0, torch.gather(want["lp"], 1, idx.clamp(min=0)), -math.inf)
        # relative to log p as the token's; -inf equals -inf
        ref.assert_within(top_lp, there, ref.d_bound(V) + 4 * ref.U * there.abs().nan_to_num(0.0, posinf=0.0),
                          "alternatives")
    else:
        assert top_lp is None and top_tok is None


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 33), (4, 255), (1, 2047), (3, 2048), (2, 2049), (7, 4099), (33, 32003),
          (1, 32768), (9, 50001), (2, 131072), (65, 4096), (300, 1000), (1, 262147),
          (513, 1500), (600, 3000), (520, 33001), (300, 70001), (257, 12000)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,V", SHAPES)
def test_forward(n, V, dtype):
    for i, (k, kind) in enumerate([(0, "none"), (1, "one"), (5, "rows"), (20, "none"), (64, "rows")]):
        z, gen = ref.random_logits(n, V, dtype, 17 * n + V + i)
        _check_forward(z, _tokens(n, V, gen), _temperature(kind, n, gen), min(k, V))


@pytest.mark.parametrize("n,V", [(5, 333), (600, 5001), (3, 70001)])
def test_what_is_wanted(n, V):
    """Every choice of outputs gives the same values."""
    z, gen = ref.random_logits(n, V, F32, 5)
    token = _tokens(n, V, gen)
    full = lmh.lmhead_logprobs(z, token, n_top=3)
    for k in (0, 3):
        for lp in (None, False):
            for ent in (None, False):
                for rank in (None, False):
                    got = lmh.lmhead_logprobs(z, token, n_top=k, logprob=lp, entropy=ent, rank=rank)
                    for g, f in zip(got[:3], full[:3]):
                        assert g is None or torch.equal(g, f)
                    assert [g is None for g in got[:3]] == [lp is False, ent is False, rank is False]
                    assert torch.equal(got[5], full[5])
                    assert (got[3] is None) == (k == 0)
    none = lmh.lmhead_logprobs(z, n_top=3)
    assert none[0] is None and none[2] is None
    assert torch.equal(none[1], full[1]) and torch.equal(none[3], full[3]) and torch.equal(none[4], full[4])
    _check_forward(z, None, None, 3, none)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("times", [1, 50, 100])
@pytest.mark.parametrize("V", [70, 700, 2048, 9001, 40000])
def test_equal_logits(V, times, dtype):
    """Ties, within a wave, across segments and more than any list holds; the rows
    repeated for the plans of larger batches."""
    n = 6
    z = ref.padded(n, V, dtype)
    gen = torch.Generator(device="cuda").manual_seed(V)
    z[0] = 1.5                                     # all equal
    z[1] = (torch.arange(V, device="cuda") % 3).to(dtype)
    z[2] = torch.randint(-2, 3, (V,), device="cuda", generator=gen).to(dtype)
    z[3] = -0.0
    z[3, ::2] = 0.0                                # zeros of both signs are equal
    z[4] = -math.inf
    z[4, V // 2] = 3.0                             # one column left
    z[5] = torch.where(torch.arange(V, device="cuda") < V - 20, -5.0, 2.0).to(dtype)
    token = torch.tensor([V - 1, V // 2, V - 2, 1, V // 2, V - 1], dtype=torch.int32, device="cuda")
    z = ref.repad(z.repeat(times, 1))
    for k in (1, 7, 64):
        _check_forward(z, token.repeat(times), None, k)
    _check_forward(z, torch.zeros(n * times, dtype=torch.int32, device="cuda"), None, 33)


@pytest.mark.parametrize("V", [5, 40, 2500, 40000, 70000])
def test_masks_and_bad_rows(V):
    """Masked columns, rows without anything, NaN, infinities, tokens that are no
    columns, temperatures that are none."""
    lowest = torch.finfo(F32).min
    z, gen = ref.random_logits(8, V, F32, 3)
    z[0, 1:] = -math.inf
    z[1, : V - 1] = lowest
    z[2] = lowest                                  # uniform over masks
    z[3, ::2] = lowest
    z[3, 1::2] = -math.inf
    z[4, V // 2:] = -math.inf
    token = torch.tensor([0, V - 1, V // 2, 0, V - 1, -100, V // 3, 0], dtype=torch.int32, device="cuda")
    k = min(V, 6)
    _check_forward(z, token, None, k)
    # rows that are NaN do not reach the others
    bad = ref.repad(z)
    bad[0] = -math.inf
    bad[2, V // 2] = math.nan
    bad[5, 0] = math.inf
    bad[7] = math.nan
    token2 = token.clone()
    token2[1], token2[3], token2[6] = V, -1, 2 ** 31 - 1
    got = lmh.lmhead_logprobs(bad, token2, n_top=k)
    for i in (0, 2, 5, 7):
        assert torch.isnan(got[1][i]) and torch.isnan(got[3][i]).all() and (got[4][i] == -1).all()
        assert (got[0][i] == 0 if i == 5 else torch.isnan(got[0][i])) and got[2][i] == -1
    for i in (1, 3, 6):
        assert torch.isnan(got[0][i]) and got[2][i] == -1 and torch.isfinite(got[1][i])
    good = torch.tensor([1, 3, 4, 6], device="cuda")
    want = lmh.lmhead_logprobs(ref.repad(z[good]), token[good], n_top=k)
    for a, b in zip((got[1], got[3], got[4]), (want[1], want[3], want[4])):
        assert torch.equal(a[good], b)
    # temperatures
    t = torch.tensor([1.0, 0.0, -1.0, math.nan, math.inf, 1e-3, 1e3, 1.0], device="cuda")
    got = lmh.lmhead_logprobs(z, token, temperature=t, n_top=k)
    for i in (1, 2, 3, 4):
        assert torch.isnan(got[1][i]) and torch.isnan(got[0][i]) and (got[4][i] == -1).all()
    rows = torch.tensor([0, 5, 6, 7], device="cuda")
    _check_forward(z[rows], token[rows], t[rows], k, tuple(x[rows] for x in got))


def test_many_parts_of_equal_logits():
    """A row in so many parts that their lists pass what is ranked at once, and a
    workspace whose contents do not matter."""
    n, V, k = 2, 4_500_003, 64
    for dtype in (F32, BF16):
        z = ref.padded(n, V, dtype)
        z[0] = 2.5
        z[1] = -math.inf
        z[1, V - 100:] = -1.0
        z[1, 7] = -2.0
        token = torch.tensor([V - 1, 7], dtype=torch.int32, device="cuda")
        ws = torch.full((lmh.lmhead_logprobs_workspace_bytes(n, V, k),), 255, dtype=torch.uint8, device="cuda")
        assert ws.numel() > 2048 * 8 * n
        got = lmh.lmhead_logprobs(z, token, n_top=k, workspace=ws)
        assert got[4][0].tolist() == list(range(k)) and got[4][1].tolist() == list(range(V - 100, V - 100 + k))
        assert got[2].tolist() == [V - 1, 100]
        _check_forward(z, token, None, k, got)
        ws.fill_(255)
        assert torch.equal(lmh.lmhead_logprobs(z, token, workspace=ws)[5], got[5])


def test_two_streams_at_once():
    """Calls on two streams, a workspace each."""
    z, gen = ref.random_logits(3, 200003, F32, 5)
    token = _tokens(3, 200003, gen)
    want = lmh.lmhead_logprobs(z, token, n_top=9)
    g = torch.randn(3, device="cuda", generator=gen)
    grad = lmh.lmhead_logprobs_bwd(z, want[5], token, g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for st in streams:
            res = lmh.lmhead_logprobs(z, token, n_top=9, stream=st)
            got.append((*res, lmh.lmhead_logprobs_bwd(z, res[5], token, g, stream=st)))
    torch.cuda.synchronize()
    for res in got:
        for a, b in zip(res, (*want, grad)):
            assert torch.equal(a, b)


def test_more_rows_than_one_launch_takes():
    """2^21 rows a launch of the forward, 2^24 of the gradient."""
    V = 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = 2 ** 24 + 3
    z = torch.randn(n, V, device="cuda", generator=gen)
    token = torch.randint(0, V, (n,), device="cuda", generator=gen).int()
    t = 0.5 + torch.rand(n, device="cuda", generator=gen)
    g = torch.randn(n, device="cuda", generator=gen)
    got = lmh.lmhead_logprobs(z, token, temperature=t, n_top=2)
    grad = lmh.lmhead_logprobs_bwd(z, got[5], token, g, dentropy=g, temperature=t)
    for lo in (0, 2 ** 21 - 2, 2 ** 23 - 2, n - 6):
        s = slice(lo, lo + 6)
        _check_forward(z[s], token[s], t[s], 2, tuple(x[s] for x in got))
        want, tol = ref.logprobs_grad(z[s], token[s], t[s], g[s], g[s])
        ref.assert_grad(grad[s], want, tol, lo)
    # every row, against the next ones: nothing was left out
    lp = torch.log_softmax(z / t[:, None], 1)
    assert torch.allclose(got[0], torch.gather(lp, 1, token.long()[:, None])[:, 0], atol=1e-5)
    assert (grad.abs().sum(1) > 0).all() and (grad.sum(1).abs() < 1e-4).all()


def test_long_rows_and_many():
    """Offsets past 2^31 elements and rows past what a short grid holds."""
    V, n = 131072, 16500                           # 2.16e9 elements
    z = torch.zeros(n, V, dtype=BF16, device="cuda")
    token = torch.full((n,), V - 1, dtype=torch.int32, device="cuda")
    z[n - 1, V - 1] = 4.0
    z[n - 1, 77] = 5.0
    lp, ent, rank, top_lp, top_tok, stats = lmh.lmhead_logprobs(z, token, n_top=3)
    assert top_tok[n - 1].tolist() == [77, V - 1, 0] and top_tok[0].tolist() == [0, 1, 2]
    assert rank[n - 1] == 1 and rank[0] == V - 1
    assert torch.allclose(lp[: n - 1], torch.full((n - 1,), -math.log(V), device="cuda"), atol=1e-5)
    _check_forward(z[n - 2:], token[n - 2:], None, 3,
                   tuple(t[n - 2:] for t in (lp, ent, rank, top_lp, top_tok, stats)))
    g = lmh.lmhead_logprobs_bwd(z, stats, token, torch.ones(1, device="cuda"), in_place=True)
    assert g is z
    want = 1.0 - math.exp(4.0 - 5.0 - float(torch.log(stats[n - 1, 1])))
    assert abs(float(g[n - 1, V - 1]) - want) < 2.0 ** -8
    assert abs(float(g[n - 2, V - 1]) - 1.0) < 2.0 ** -8


@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,V", [(1, 1), (3, 2), (2, 7), (5, 33), (3, 4095), (2, 4097), (7, 8200), (33, 32003),
                                 (2, 131072), (300, 1000)])
def test_gradient(n, V, dtype, grad):
    for i, kind in enumerate(["none", "one", "rows"]):
        z, gen = ref.random_logits(n, V, dtype, 31 * n + V + i)
        token = _tokens(n, V, gen)
        t = _temperature(kind, n, gen)
        stats = lmh.lmhead_logprobs(z, token, temperature=t)[5]
        g = torch.randn(n, device="cuda", generator=gen)
        h = 0.3 * torch.randn(n, device="cuda", generator=gen)
        g[n // 2] = 0.0
        for dg, dh in ((g, h), (g, None), (None, h), (g[:1], h[:1]), (None, None)):
            out = ref.padded(n, V, grad)
            got = lmh.lmhead_logprobs_bwd(z, stats, token, dg, dentropy=dh, temperature=t, dlogits=out)
            assert got is out and ref.padding_holds(out)
            want, tol = ref.logprobs_grad(z, token, t, dg, dh)
            ref.assert_grad(got, want, tol, (kind, dg is None, dh is None))
        if dtype == grad:
            want = lmh.lmhead_logprobs_bwd(z, stats, token, g, dentropy=h, temperature=t, grad_dtype=grad)
            zz = ref.padded(n, V, dtype)
            zz.copy_(z)
            got = lmh.lmhead_logprobs_bwd(zz, stats, token, g, dentropy=h, temperature=t, in_place=True)
            assert got is zz and torch.equal(got, want) and ref.padding_holds(zz)


@pytest.mark.parametrize("V", [5, 2500, 70000])
def test_gradient_of_masks_and_bad_rows(V):
    lowest = torch.finfo(F32).min
    z, gen = ref.random_logits(9, V, F32, 4)
    z[0, 1:] = -math.inf
    z[1, : V - 1] = lowest
    z[2] = lowest
    z[3, ::2] = lowest
    z[3, 1::2] = -math.inf
    z[4, V // 2:] = -math.inf
    token = torch.tensor([0, V - 1, V // 2, 0, V - 1, -100, V // 3, 0, 1], dtype=torch.int32, device="cuda")
    g = torch.randn(9, device="cuda", generator=gen)
    h = torch.randn(9, device="cuda", generator=gen)
    stats = lmh.lmhead_logprobs(z, token)[5]
    got = lmh.lmhead_logprobs_bwd(z, stats, token, g, dentropy=h)
    want, tol = ref.logprobs_grad(z, token, None, g, h)
    ref.assert_grad(got, want, tol, "masks")
    # bad rows: NaN where asked for, zeros where nothing is
    bad = ref.repad(z)
    bad[0] = -math.inf
    bad[2, 1] = math.nan
    bad[6] = math.inf
    bad[7, 0] = math.nan
    t2 = token.clone()
    t2[4] = V
    g2, h2 = g.clone(), h.clone()
    g2[7] = h2[7] = 0.0
    g2[4] = 0.0
    stats = lmh.lmhead_logprobs(bad, t2)[5]
    got = lmh.lmhead_logprobs_bwd(bad, stats, t2, g2, dentropy=h2)
    for i in (0, 2, 4, 6):
        assert torch.isnan(got[i]).all(), i
    assert (got[7] == 0).all()
    keep = torch.tensor([1, 3, 5, 8], device="cuda")
    ref.assert_grad(got[keep], want[keep], tol[keep], "beside bad rows")


def test_gradient_against_differences():
    """Central differences of the 64-bit log-probability and entropy."""
    n, V, eps = 4, 1031, 1e-4
    z, gen = ref.random_logits(n, V, F32, 8, sigma=1.5)
    token = torch.tensor([3, 1030, 512, 77], dtype=torch.int32, device="cuda")
    t = 0.7 + 0.6 * torch.rand(n, device="cuda", generator=gen)
    g = torch.randn(n, device="cuda", generator=gen)
    h = torch.randn(n, device="cuda", generator=gen)
    got = lmh.lmhead_logprobs_bwd(z, lmh.lmhead_logprobs(z, token, temperature=t)[5], token, g, dentropy=h,
                                  temperature=t)
    cols = [0, 3, 77, 511, 512, 1029, 1030]

    def value(w):
        r = ref.logprobs(w, token, t)
        return g.double() * r["logprob"] + h.double() * r["entropy"]

    for j in cols:
        up, down = z.double().clone(), z.double().clone()
        up[:, j] += eps
        down[:, j] -= eps
        diff = (value(up) - value(down)) / (2 * eps)
        # the third derivative times eps^2 / 6 is below 1e-7 here
        assert torch.allclose(got[:, j].double(), diff, rtol=1e-5, atol=1e-6), j


def test_runs_are_equal_and_any_row_order():
    """Bitwise the same twice; a row's result does not depend on the batch."""
    z, gen = ref.random_logits(700, 9001, F32, 21)
    token = _tokens(700, 9001, gen)
    a = lmh.lmhead_logprobs(z, token, n_top=9)
    b = lmh.lmhead_logprobs(z, token, n_top=9)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    one = lmh.lmhead_logprobs(z[650:651], token[650:651], n_top=9)
    for x, y in zip(a[:5], one[:5]):
        assert torch.allclose(x[650:651].double(), y.double(), rtol=1e-6, atol=1e-5)
    assert torch.equal(a[4][650:651], one[4]) and torch.equal(a[2][650:651], one[2])


def test_empty_batch():
    z = torch.empty(0, 64, device="cuda")
    got = lmh.lmhead_logprobs(z, torch.empty(0, dtype=torch.int32, device="cuda"), n_top=2)
    assert [tuple(t.shape) for t in got] == [(0,), (0,), (0,), (0, 2), (0, 2), (0, 4)]
    g = lmh.lmhead_logprobs_bwd(z, got[5], None, None)
    assert g.shape == (0, 64)


def test_a_row_of_its_own():
    """One row needs no pitch: any vocabulary size, contiguous."""
    for V in (1, 5, 50257):
        for dtype in (F32, BF16):
            z = torch.randn(1, V, device="cuda").to(dtype)
            token = torch.tensor([V // 2], dtype=torch.int32, device="cuda")
            got = lmh.lmhead_logprobs(z, token, n_top=min(V, 3))
            _check_forward(z, token, None, min(V, 3), got)
            g = torch.ones(1, device="cuda")
            want, tol = ref.logprobs_grad(z, token, None, g, None)
            ref.assert_grad(lmh.lmhead_logprobs_bwd(z, got[5], token, g), want, tol, V)
            lmh.lmhead_logprobs_bwd(z, got[5], token, g, in_place=True)
            ref.assert_within(z, want, tol + ref.HALF[dtype] * want.abs() * 1.01, "in place")


def test_given_outputs_and_streams():
    z, gen = ref.random_logits(40, 5000, F32, 2)
    token = _tokens(40, 5000, gen)
    want = lmh.lmhead_logprobs(z, token, n_top=4)
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(lmh.lmhead_logprobs_workspace_bytes(40, 5000, 4), dtype=torch.uint8, device="cuda")
    got = lmh.lmhead_logprobs(z, token, -100, None, 4, *outs, workspace=ws)
    for g, o, w in zip(got, outs, want):
        assert g is o and torch.equal(g, w)
    side = torch.cuda.Stream()
    dg = torch.ones(1, device="cuda")
    grad = lmh.lmhead_logprobs_bwd(z, want[5], token, dg)
    torch.cuda.synchronize()
    for st in (side, side.cuda_stream):
        got = lmh.lmhead_logprobs(z, token, n_top=4, workspace=ws, stream=st)
        g2 = lmh.lmhead_logprobs_bwd(z, want[5], token, dg, stream=st)
        torch.cuda.synchronize()
        for g, w in zip((*got, g2), (*want, grad)):
            assert torch.equal(g, w)
    with pytest.raises(ValueError):
        lmh.lmhead_logprobs(z, token, stream=side.cuda_stream)


def test_captured_policy_gradient_step():
    """Forward, an advantage from it, backward and the GEMMs, captured and
    replayed on other inputs."""
    M, K, V = 48, 128, 4104
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    W = (0.1 * torch.randn(V, K, device="cuda", generator=gen)).bfloat16()
    token = torch.randint(0, V, (M,), device="cuda", generator=gen).int()
    old = torch.full((M,), -8.0, device="cuda")
    adv = torch.randn(M, device="cuda", generator=gen)
    bonus = torch.full((1,), 0.01, device="cuda")

    def step():
        z = lmh.lmhead_logits(x, W, out_dtype="fp32")
        lp, ent, _, _, _, stats = lmh.lmhead_logprobs(z, token, rank=False)
        g = -adv * torch.exp(lp - old)
        dz = lmh.lmhead_logprobs_bwd(z, stats, token, g, dentropy=bonus, grad_dtype="bf16")
        return lp, ent, lmh.lmhead_dgrad(dz, W, dx_dtype="fp32"), lmh.lmhead_wgrad(dz, x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(torch.randn(M, K, device="cuda", generator=gen))
        token.copy_(torch.randint(0, V, (M,), device="cuda", generator=gen))
        adv.copy_(torch.randn(M, device="cuda", generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b), i
