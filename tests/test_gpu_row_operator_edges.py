"""Log-probabilities and distillation at the edges of what the calls take: rows
that ask for nothing, and temperatures at the ends of their range."""
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
