"""Log-probabilities and distillation at the edges of what the calls take: rows
that ask for no gradient, the smallest temperatures, logits with a large common
part, and entropy gradients that are large per unit of temperature."""
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


def _lists(n, V, gen):
    ids = torch.stack([torch.randperm(V, device="cuda", generator=gen)[:5] for _ in range(n)]).int()
    return ids, torch.log_softmax(torch.randn(n, 5, device="cuda", generator=gen), 1) - 0.3


# One size for each way in which loss and gradient are computed together: rows in the
# registers of 256, 512 or 1024 threads (a larger batch takes half as many for the
# third), and rows read twice.
@pytest.mark.parametrize("n,V", [(6, 12), (6, 9001), (6, 20000), (300, 20000), (6, 40000), (6, 70000)])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,grad", [(F32, F32), (BF16, BF16)])
def test_no_gradient_from_above_at_any_temperature(n, V, dtype, grad, tail):
    """A padded row has no upstream gradient, and often no temperature either: its
    gradient is zero, while its loss is NaN.  With one it is NaN."""
    z, gen = ref.random_logits(n, V, dtype, 3 * V + n)
    ids, vals = _lists(n, V, gen)
    T = torch.full((n,), 0.8, device="cuda")
    T[:5] = torch.tensor([0.0, -1.0, math.nan, math.inf, 0.0], device="cuda")
    dloss = torch.randn(n, device="cuda", generator=gen)
    dloss[:4] = torch.tensor([0.0, -0.0, 0.0, 0.0], device="cuda")
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail, temperature=T)
    dz = lmh.lmhead_distill_bwd(z, stats, ids, vals, dloss, tail=tail, temperature=T, grad_dtype=grad)
    fused = lmh.lmhead_distill_fused(z, ids, vals, dloss, tail=tail, temperature=T, grad_dtype=grad)
    want = ref.distill(z[5:], ids[5:], vals[5:], tail, T[5:], dloss[5:])
    for got_loss, got in ((loss, dz), fused[::2]):
        assert torch.isnan(got_loss[:5]).all()
        assert (got[:4] == 0).all() and torch.isnan(got[4]).all()
        ref.assert_grad(got[5:], want["dlogits"], want["tol_dlogits"], "beside them")
    token = ids[:, 0].contiguous()
    stats = lmh.lmhead_logprobs(z, token, temperature=T)[5]
    h = dloss.clone()
    got = lmh.lmhead_logprobs_bwd(z, stats, token, dloss, dentropy=h, temperature=T, grad_dtype=grad)
    assert (got[:4] == 0).all() and torch.isnan(got[4]).all()
    want, tol = ref.logprobs_grad(z[5:], token[5:], T[5:], dloss[5:], h[5:])
    ref.assert_grad(got[5:], want, tol, "beside them")
    zero = torch.zeros(1, device="cuda")
    assert (lmh.lmhead_distill_fused(z, ids, vals, zero, tail=tail, temperature=T)[2] == 0).all()


def test_padded_rows_leave_the_weights_gradient_alone():
    """Rows without gradient and temperature add nothing to dW."""
    M, K, V = 16, 64, 1000
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    W = (0.2 * torch.randn(V, K, device="cuda", generator=gen)).bfloat16()
    z = lmh.lmhead_logits(x, W, out_dtype="fp32")
    ids, vals = _lists(M, V, gen)
    T, up = torch.ones(M, device="cuda"), torch.full((M,), 1.0 / 11, device="cuda")
    T[11:], up[11:] = 0.0, 0.0
    dz = lmh.lmhead_distill_fused(z, ids, vals, up, temperature=T, grad_dtype="bf16")[2]
    short = lmh.lmhead_distill_fused(z[:11], ids[:11], vals[:11], up[:11], temperature=T[:11], grad_dtype="bf16")[2]
    assert torch.equal(dz[:11], short) and (dz[11:] == 0).all()
    dW = lmh.lmhead_wgrad(dz, x)
    want = dz[:11].double().t() @ x[:11].double()
    # M FP32 additions of products of two BF16 values, exact in FP32
    assert ((dW - want).abs() <= M * ref.U * (dz[:11].double().abs().t() @ x[:11].double().abs()) + ref.TINY).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [4, 200, 70000])
def test_the_smallest_temperatures(V, tail):
    """From where log2(e) / T passes FP32 (4.24e-39) a row is NaN in every call, with
    every column listed too; above that it is the largest logits' columns alone."""
    none = [1e-45, 1e-39, 2.9e-39, 4e-39, 4.2e-39]
    T = torch.tensor(none + [4.3e-39, 1e-38, 2e-38], device="cuda")
    n, bad = T.numel(), len(none)
    assert (T > 0).all()
    z = ref.padded(n, V, F32)
    z.fill_(1.5)
    z[:, 2] = 0.25
    token = torch.zeros(n, dtype=torch.int32, device="cuda")
    k = min(V, 256)
    lp, ent, rank, top_lp, top_tok, stats = lmh.lmhead_logprobs(z, token, temperature=T, n_top=3)
    one = torch.ones(1, device="cuda")
    g = lmh.lmhead_logprobs_bwd(z, stats, token, one, dentropy=0.0 * one, temperature=T)
    assert torch.isnan(lp[:bad]).all() and torch.isnan(ent[:bad]).all() and (rank[:bad] == -1).all()
    assert torch.isnan(top_lp[:bad]).all() and (top_tok[:bad] == -1).all() and torch.isnan(g[:bad]).all()
    log_n = math.log(V - 1)
    for got in (-lp[bad:], ent[bad:], -top_lp[bad:, 0], -top_lp[bad:, 2]):
        assert ((got.double() - log_n).abs() <= ref.d_bound(V) + 4 * ref.U * log_n).all()
    assert top_tok[bad:].tolist() == [[0, 1, 3]] * (n - bad) and (rank[bad:] == 0).all()
    # The teacher gives the lesser column nothing (exp(-1000) is 0 in 64 bits): with any
    # share its loss would pass FP32.
    ids = torch.arange(k, dtype=torch.int32, device="cuda").expand(n, k).contiguous()
    vals = torch.full((n, k), math.log(0.5 / k), device="cuda")
    vals[:, 2] = -math.inf if not tail else -1000.0
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail, temperature=T)
    dz = lmh.lmhead_distill_bwd(z, stats, ids, vals, one, tail=tail, temperature=T)
    fused = lmh.lmhead_distill_fused(z, ids, vals, one, tail=tail, temperature=T)
    for got_loss, got in ((loss, dz), fused[::2]):
        assert torch.isnan(got_loss[:bad]).all() and torch.isnan(got[:bad]).all()
        assert torch.isfinite(got_loss[bad:]).all() and torch.isfinite(got[bad:]).all()
        assert (got[bad:, 2] == 0).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,V", [(6, 50), (6, 5000), (300, 20000), (6, 40000), (6, 70000), (600, 900)])
def test_logits_with_a_large_common_part(n, V, dtype, tail):
    """Rows of masks only (all at the type's lowest value), of one large value, of ties
    at a low temperature: the loss is that of the same row about zero."""
    z, gen = ref.random_logits(n, V, dtype, V + n)
    z[0] = torch.finfo(dtype).min
    z[1] = 1e30
    z[2] = 0.1
    z[3] = -3e38
    z[4] = torch.finfo(dtype).min
    z[4, 1] = -2.0 ** 127                  # the listed columns' largest: one term alone
    T = torch.ones(n, device="cuda")
    T[2] = 1e-15
    ids = torch.arange(7, device="cuda").expand(n, 7).int().contiguous()
    vals = torch.log_softmax(torch.randn(n, 7, device="cuda", generator=gen), 1) - 0.3
    dloss = torch.randn(n, device="cuda", generator=gen)
    want = ref.distill(z, ids, vals, tail, T, dloss)
    plain = z.clone()
    plain[:4] = 0.0
    T1 = torch.ones(n, device="cuda")
    if tail:                               # q does not depend on T
        same = ref.distill(plain[:4], ids[:4], vals[:4], tail, T1[:4], dloss[:4])
        assert torch.allclose(same["loss"], want["loss"][:4], rtol=1e-12)
    assert torch.isfinite(want["loss"]).all() and (want["loss"][:4] < 20).all()
    if tail:
        # The reference forms the others' shares of p_r from log p - log p_r, whose log(V - 7)
        # is lost beside 1.7e38: of row 4 they are 1 / (V - 7) each, and p is column 1's.
        q = torch.exp(vals[4].double())
        q_r = 1.0 - q.sum()
        row = torch.full((V,), -float(q_r) / (V - 7), dtype=torch.float64, device="cuda")
        row[:7] = -q
        row[1] += 1.0
        want["dlogits"][4] = row * dloss[4].double()
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail, temperature=T)
    dz = lmh.lmhead_distill_bwd(z, stats, ids, vals, dloss, tail=tail, temperature=T)
    fused = lmh.lmhead_distill_fused(z, ids, vals, dloss, tail=tail, temperature=T)
    for got_loss, got in ((loss, dz), fused[::2]):
        ref.assert_within(got_loss, want["loss"], want["tol_loss"], "loss")
        ref.assert_grad(got, want["dlogits"], want["tol_dlogits"], "dlogits")


@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [6, 5000])
def test_entropy_gradient_at_low_temperatures(V, dtype, grad):
    """Where p is 0 the entropy has no gradient, however large h / T is."""
    z, gen = ref.random_logits(6, V, dtype, V)
    token = torch.randint(0, V, (6,), device="cuda", generator=gen).int()
    T = torch.tensor([1e-37, 1e-38, 4e-37, 1e-36, 1e-3, 1.0], device="cuda")
    z[2, :2] = 40.0                        # an even pair: entropy log 2
    g = torch.full((6,), 0.25, device="cuda")
    h = torch.tensor([1.0, -0.5, 1.0, 50.0, 1e35, 3e37], device="cuda")
    for dlogprob in (g, None):
        stats = lmh.lmhead_logprobs(z, token, temperature=T)[5]
        got = lmh.lmhead_logprobs_bwd(z, stats, token, dlogprob, dentropy=h, temperature=T, grad_dtype=grad)
        assert torch.isfinite(got).all()
        want, tol = ref.logprobs_grad(z, token, T, dlogprob, h)
        ref.assert_grad(got, want, tol, "dlogits")
