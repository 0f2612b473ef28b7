"""Log-probabilities and distillation at sizes that reach each way in which the
library shares out rows, with both types of logits where rows are masked or bad."""
import math

import pytest
import torch

import lm_head_fp32_amd as lmh
import row_reference as ref
from test_gpu_distill import _check, _lists

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


# Forward: 8 waves to a row (257 - 511 rows of more than 8192 columns, fewer rows of 8193 -
# 16384), 16 (one part and several), several parts of 4 waves.  Loss and gradient together:
# 256, 512 and 1024 threads of 32 values, 512 and 1024 of 64.
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,grad", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("n,V,k", [(300, 32003, 20), (257, 20001, 70), (300, 12000, 33), (5, 9001, 9),
                                   (256, 16385, 256), (257, 32768, 64), (20, 16384, 5), (511, 8193, 3),
                                   (129, 40001, 17)])
def test_distillation(n, V, k, dtype, grad, tail):
    z, gen = ref.random_logits(n, V, dtype, n + V + k)
    T = 0.7 + 1.5 * torch.rand(n, device="cuda", generator=gen)
    ids, vals = _lists(z, k, tail, F32, gen, T=T)
    _check(z, ids, vals, tail, T, torch.randn(n, device="cuda", generator=gen), grad)


@pytest.mark.parametrize("tail", [False, True])
def test_distillation_of_many_rows_in_parts(tail):
    n, V, k = 520, 262200, 40
    z, gen = ref.random_logits(n, V, BF16, 5)
    assert lmh.lmhead_distill_workspace_bytes(n, V) > 0
    ids, vals = _lists(z, k, tail, F32, gen)
    up = torch.randn(n, device="cuda", generator=gen)
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail)
    g = lmh.lmhead_distill_bwd(z, stats, ids, vals, up, tail=tail, grad_dtype=F32)
    for lo in range(0, n, 65):  # the reference's tables in 64 bits, by rows
        s = slice(lo, min(lo + 65, n))
        want = ref.distill(z[s], ids[s], vals[s], tail, None, up[s])
        ref.assert_within(loss[s], want["loss"], want["tol_loss"], "loss")
        ref.assert_grad(g[s], want["dlogits"], want["tol_dlogits"], "dlogits")


def test_more_rows_than_one_launch_of_the_gradient_takes():
    """2^24 rows a launch."""
    n, V = 2 ** 24 + 3, 8
    gen = torch.Generator(device="cuda").manual_seed(4)
    z = torch.randn(n, V, device="cuda", generator=gen)
    ids = torch.randint(0, V, (n, 2), device="cuda", generator=gen).int()
    vals = torch.log_softmax(torch.randn(n, 2, device="cuda", generator=gen), 1) - 0.5
    T = 0.5 + torch.rand(n, device="cuda", generator=gen)
    up = 0.5 + torch.rand(n, device="cuda", generator=gen)
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=True, temperature=T)
    g = lmh.lmhead_distill_bwd(z, stats, ids, vals, up, tail=True, temperature=T)
    for lo in (0, 2 ** 21 - 2, 2 ** 23 - 2, n - 6):
        s = slice(lo, lo + 6)
        want = ref.distill(z[s], ids[s], vals[s], True, T[s], up[s])
        ref.assert_within(loss[s], want["loss"], want["tol_loss"], lo)
        ref.assert_grad(g[s], want["dlogits"], want["tol_dlogits"], lo)
    # every row: nothing was left out, and a gradient of p sums to zero
    assert (g.abs().sum(1) > 0).all() and (g.sum(1).abs() < 1e-4).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("times", [1, 30])
@pytest.mark.parametrize("dtype,grad", [(F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("V", [13, 3001, 12001, 20003, 32768, 40000, 70000])
def test_masked_and_bad_rows(V, dtype, grad, times, tail):
    """Masked columns and rows, lists with nothing, NaN and infinities, tokens that are no
    columns, beside rows that are right; the rows repeated for the plans of larger batches."""
    lowest = torch.finfo(dtype).min
    n, k = 13, 5
    z, gen = ref.random_logits(n, V, dtype, 9 + V)
    ids, vals = _lists(z, k, tail, F32, gen, ragged=False)
    ids[:] = torch.tensor([1, 2, 7, 11, 5], device="cuda", dtype=torch.int32)
    if tail:
        vals = torch.log_softmax(vals, 1) - 0.2
    z[0, 8:] = lowest
    z[1, 8:] = -math.inf
    z[1, 11], z[1, 9] = 0.5, 1.0
    ids[2] = -1
    vals[3] = -math.inf
    z[4, 2] = -math.inf                  # a listed column with q > 0
    z[5] = lowest
    ids[6, 1:] = ids[6, 0]               # one token, five times
    dloss = torch.randn(n, device="cuda", generator=gen)
    ok = list(range(7))
    want = ref.distill(z[ok], ids[ok], vals[ok], tail, None, dloss[ok])
    z[2] = math.nan                      # of no list: not looked at
    z[7, 3] = math.nan
    z[8, V - 1] = math.inf
    z[9] = -math.inf
    ids[10, 2] = V
    vals[11, 1] = math.nan
    vals[12, 0] = math.inf
    z = ref.repad(z.repeat(times, 1))
    ids, vals, dloss = ids.repeat(times, 1), vals.repeat(times, 1), dloss.repeat(times)
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail)
    g = lmh.lmhead_distill_bwd(z, stats, ids, vals, dloss, tail=tail, grad_dtype=grad)
    fused = lmh.lmhead_distill_fused(z, ids, vals, dloss, tail=tail, grad_dtype=grad)
    for got_loss, got in ((loss, g), fused[::2]):
        for lo in range(0, n * times, n):
            a, b = got_loss[lo:lo + n], got[lo:lo + n]
            assert torch.isnan(a[7:]).all() and torch.isnan(b[7:]).all()
            ref.assert_within(a[:7], want["loss"], want["tol_loss"], "loss")
            ref.assert_grad(b[:7], want["dlogits"], want["tol_dlogits"], "dlogits")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,grad", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,V", [(300, 20000), (260, 32768), (260, 12000), (20, 20000)])
def test_tokens_listed_twice(n, V, dtype, grad, tail):
    z, gen = ref.random_logits(n, V, dtype, 6)
    k = 256
    ids = torch.randint(0, V, (n, k), device="cuda", generator=gen).int()
    ids[1::4] = V - 1
    ids[2::4, : k // 2] = ids[2::4, k // 2:]
    ids[3::4, 1:] = -1
    vals = torch.randn(n, k, device="cuda", generator=gen)
    if tail:
        vals = torch.log_softmax(vals, 1) - 0.7
    _check(z, ids, vals, tail, None, torch.randn(n, device="cuda", generator=gen), grad)


@pytest.mark.parametrize("times", [1, 30, 60])
@pytest.mark.parametrize("V", [13, 1500, 3001, 12001, 40000, 70000])
def test_log_probabilities_of_masked_and_bad_rows(V, times):
    """The same of log-probabilities and their gradient, BF16 logits."""
    lowest = torch.finfo(BF16).min
    n, k = 10, 6
    z, gen = ref.random_logits(n, V, BF16, 3 + V)
    z[0, 1:] = -math.inf
    z[1, : V - 1] = lowest
    z[2] = lowest
    z[3, ::2] = lowest
    z[3, 1::2] = -math.inf
    z[4, V // 2:] = -math.inf
    token = torch.tensor([0, V - 1, V // 2, 0, V - 1, 3, 1, 2, 0, -100], dtype=torch.int32, device="cuda")
    g, h = (torch.randn(n, device="cuda", generator=gen) for _ in range(2))
    ok = list(range(6))
    want = ref.logprobs(z[ok], token[ok], None)
    idx, val = ref.top(z[ok], k)
    want_g, tol_g = ref.logprobs_grad(z[ok], token[ok], None, g[ok], h[ok])
    z[6, V // 2] = math.nan
    z[7, 0] = math.inf
    z[8] = -math.inf
    z[9, V - 1] = math.nan
    z = ref.repad(z.repeat(times, 1))
    token, g, h = token.repeat(times), g.repeat(times), h.repeat(times)
    lp, ent, rank, top_lp, top_tok, stats = lmh.lmhead_logprobs(z, token, n_top=k)
    dz = lmh.lmhead_logprobs_bwd(z, stats, token, g, dentropy=h, grad_dtype=F32)
    there = torch.where(idx >= 0, torch.gather(want["lp"], 1, idx.clamp(min=0)), -math.inf)
    tol = ref.d_bound(V) + 4 * ref.U * there.abs().nan_to_num(0.0, posinf=0.0)
    for lo in range(0, n * times, n):
        s = slice(lo, lo + 6)
        ref.assert_within(lp[s], want["logprob"], want["tol_logprob"], "logprob")
        ref.assert_within(ent[s], want["entropy"], want["tol_entropy"], "entropy")
        assert torch.equal(rank[s], want["rank"]) and torch.equal(top_tok[s].long(), idx)
        ref.assert_within(top_lp[s], there, tol, "alternatives")
        ref.assert_grad(dz[s], want_g, tol_g, "dlogits")
        s = slice(lo + 6, lo + n)
        assert torch.isnan(ent[s]).all() and (rank[s] == -1).all()
        assert torch.isnan(top_lp[s]).all() and (top_tok[s] == -1).all() and torch.isnan(dz[s]).all()
        assert torch.isnan(lp[lo + 6:lo + 9]).all() and lp[lo + 9] == 0
