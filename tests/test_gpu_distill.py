"""Distillation from a teacher's listed tokens: loss and gradient against the
definitions in 64 bits (tests/row_reference.py)."""
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


def _lists(z, k, tail, vdtype, gen, ragged=True, T=None):
    """Distinct tokens of each row in random order, with a teacher's values."""
    n, V = z.shape
    t = 0.6 * z.float() + torch.randn(n, V, device="cuda", generator=gen)
    t = torch.where(torch.isfinite(t), t, -20.0)
    ids = torch.argsort(torch.rand(n, V, device="cuda", generator=gen), dim=1)[:, :k]
    if k > 1:  # the likeliest among them
        ids[:, 0] = t.argmax(1)
        dup = (ids[:, 1:] == ids[:, :1])
        ids[:, 1:][dup] = -1
    vals = torch.gather(t, 1, ids.clamp(min=0))
    if tail:
        Td = 1.0 if T is None else T.reshape(-1, 1)
        vals = vals / Td - torch.logsumexp(t / Td, 1, keepdim=True)
    if ragged and n > 1:
        length = torch.randint(0, k + 1, (n, 1), device="cuda", generator=gen)
        length[0] = 0
        gone = torch.arange(k, device="cuda")[None] >= length
        ids = torch.where(gone & (torch.arange(n, device="cuda") % 2 == 0)[:, None], -1, ids)
        vals = torch.where(gone & (torch.arange(n, device="cuda") % 2 == 1)[:, None], -math.inf, vals)
    return ids.int().contiguous(), vals.to(vdtype).contiguous()


def _check(z, ids, vals, tail, T, dloss, grad):
    n, V = z.shape
    want = ref.distill(z, ids, vals, tail, T, dloss)
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail, temperature=T)
    ref.assert_within(loss, want["loss"], want["tol_loss"], "loss")
    assert stats.shape == (n, 8) and torch.equal(stats[:, 2].nan_to_num(7.0), loss.nan_to_num(7.0))
    out = ref.padded(n, V, grad)
    got = lmh.lmhead_distill_bwd(z, stats, ids, vals, dloss, tail=tail, temperature=T, dlogits=out)
    assert got is out and ref.padding_holds(out)
    ref.assert_grad(got, want["dlogits"], want["tol_dlogits"], "dlogits")
    out2 = ref.padded(n, V, grad)
    loss2, stats2, got2 = lmh.lmhead_distill_fused(z, ids, vals, dloss, tail=tail, temperature=T, dlogits=out2)
    assert got2 is out2 and ref.padding_holds(out2)
    ref.assert_within(loss2, want["loss"], want["tol_loss"], "fused loss")
    ref.assert_grad(got2, want["dlogits"], want["tol_dlogits"], "fused dlogits")
    # either record serves the gradient
    got3 = lmh.lmhead_distill_bwd(z, stats2, ids, vals, dloss, tail=tail, temperature=T, grad_dtype=grad)
    ref.assert_grad(got3, want["dlogits"], want["tol_dlogits"], "dlogits from the fused record")
    if z.dtype == grad:
        for fused in (False, True):
            zz = ref.padded(n, V, z.dtype)
            zz.copy_(z)
            if fused:
                _, _, g = lmh.lmhead_distill_fused(zz, ids, vals, dloss, tail=tail, temperature=T, in_place=True)
                assert torch.equal(g, got2)
            else:
                g = lmh.lmhead_distill_bwd(zz, stats, ids, vals, dloss, tail=tail, temperature=T, in_place=True)
                assert torch.equal(g, got)
            assert g is zz and ref.padding_holds(zz)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,grad", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("n,V,k", [(1, 1, 1), (3, 2, 1), (2, 7, 7), (5, 33, 4), (4, 2048, 64), (3, 2049, 256),
                                   (7, 4099, 1), (33, 32003, 16), (9, 32768, 65), (4, 50001, 20), (3, 65536, 100),
                                   (3, 65540, 33), (2, 131072, 64), (300, 1000, 10), (520, 9000, 65),
                                   (600, 1500, 20), (513, 33000, 70)])
def test_loss_and_gradient(n, V, k, dtype, grad, tail):
    for i, (kind, vdtype) in enumerate([("none", F32), ("rows", BF16), ("one", F32)]):
        z, gen = ref.random_logits(n, V, dtype, 13 * n + V + k + i)
        T = None if kind == "none" else 0.7 + 1.5 * torch.rand(n if kind == "rows" else 1, device="cuda", generator=gen)
        ids, vals = _lists(z, k, tail, vdtype, gen, T=T)
        dloss = torch.randn(n if i else 1, device="cuda", generator=gen)
        if i == 2:
            dloss[n // 2] = 0.0
        _check(z, ids, vals, tail, T, dloss, grad)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("times", [1, 150])
@pytest.mark.parametrize("V", [6, 2500, 40000, 70000])
def test_tokens_listed_twice(V, times, tail):
    """Twice, side by side and far apart, and a list of one token only; the rows
    repeated for the plan of larger batches."""
    z, gen = ref.random_logits(4 * times, V, F32, 6)
    k = 256
    ids = torch.randint(0, V, (4, k), device="cuda", generator=gen).int()
    ids[1] = V - 1
    ids[2, : k // 2] = ids[2, k // 2:]
    ids[3, 1:] = -1
    ids = ids.repeat(times, 1)
    vals = torch.randn(4 * times, k, device="cuda", generator=gen)
    if tail:
        vals = torch.log_softmax(vals, 1) - 0.7
    dloss = torch.tensor([0.5, -1.0, 2.0, 1.0], device="cuda").repeat(times)
    _check(z, ids, vals, tail, None, dloss, F32)
    for _ in range(2):
        a = lmh.lmhead_distill_fused(z, ids, vals, dloss, tail=tail)
        b = lmh.lmhead_distill_fused(z, ids, vals, dloss, tail=tail)
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("V", [9, 3001, 40000, 70000])
def test_a_tail_that_hardly_is_one(V):
    """Lists with nearly all of the student's probability, or with all columns;
    teachers whose list sums to one, or to more."""
    k = min(V - 1, 8)
    z, gen = ref.random_logits(6, V, F32, 7, sigma=1.0)
    ids = torch.arange(k, device="cuda").expand(6, k).int().contiguous()
    vals = torch.log_softmax(torch.randn(6, k, device="cuda", generator=gen), 1) - 0.01
    z[0, :k] += 30.0
    z[1, :k] += 80.0
    z[2, :k] += 120.0       # the others' share is below FP32
    vals[3] += 0.01         # sums to one, up to rounding
    vals[4] += 0.5          # to more than one
    z[5, :k] -= 120.0       # the listed ones' share is
    _check(z, ids, vals, True, None, torch.ones(1, device="cuda"), F32)
    # every other column masked: the list is all there is
    z[:, k:] = -math.inf
    _check(z, ids, vals, True, None, torch.ones(1, device="cuda"), F32)
    z[:, k:] = torch.finfo(F32).min
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=True)
    g = lmh.lmhead_distill_bwd(z, stats, ids, vals, torch.ones(1, device="cuda"), tail=True)
    assert torch.isfinite(g).all() and torch.isfinite(loss).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [12, 3001, 40000, 70000])
def test_masks_and_bad_rows(V, tail):
    lowest = torch.finfo(F32).min
    n, k = 12, 5
    z, gen = ref.random_logits(n, V, F32, 9)
    ids, vals = _lists(z, k, tail, F32, gen, ragged=False)
    ids[:, 1:] = torch.tensor([2, 7, 11, 5], device="cuda", dtype=torch.int32)
    ids[:, 0] = 1
    if tail:
        vals = torch.log_softmax(vals, 1) - 0.2
    z[0, 8:] = lowest
    z[1, 8:] = -math.inf
    z[1, 11], z[1, 9] = 0.5, 1.0
    ids[2] = -1
    vals[3] = -math.inf
    z[4, 2] = -math.inf                  # a listed column with q > 0
    dloss = torch.randn(n, device="cuda", generator=gen)
    ok = torch.tensor([0, 1, 2, 3, 4], device="cuda")
    _check(ref.repad(z[ok]), ids[ok], vals[ok], tail, None, dloss[ok], F32)
    bad = ref.repad(z)
    bids, bvals = ids.clone(), vals.clone()
    bad[5, 3] = math.nan
    bad[6, 7] = math.inf
    bad[7] = -math.inf
    bids[8, 2] = V
    bids[9, 0] = 2 ** 31 - 1
    bvals[10, 1] = math.nan
    bvals[11, 0] = math.inf
    bad[2] = math.nan                    # empty list: not read
    loss, stats = lmh.lmhead_distill_fwd(bad, bids, bvals, tail=tail)
    g = lmh.lmhead_distill_bwd(bad, stats, bids, bvals, dloss, tail=tail)
    for got_loss, got in ((loss, g), lmh.lmhead_distill_fused(bad, bids, bvals, dloss, tail=tail)[::2]):
        for i in range(5, n):
            assert torch.isnan(got_loss[i]) and torch.isnan(got[i]).all(), i
        assert got_loss[2] == 0 and (got[2] == 0).all() and got_loss[3] == 0 and (got[3] == 0).all()
        want = ref.distill(z[ok], ids[ok], vals[ok], tail, None, dloss[ok])
        ref.assert_within(got_loss[ok], want["loss"], want["tol_loss"], "beside bad rows")
        ref.assert_grad(got[ok], want["dlogits"], want["tol_dlogits"], "beside bad rows")
    zero = torch.zeros(1, device="cuda")
    assert (lmh.lmhead_distill_bwd(bad, stats, bids, bvals, zero, tail=tail) == 0).all()
    assert (lmh.lmhead_distill_fused(bad, bids, bvals, zero, tail=tail)[2] == 0).all()
    T = torch.tensor([0.0, -1.0, math.nan, math.inf, 1.0], device="cuda")
    loss, stats, g = lmh.lmhead_distill_fused(z[5:10], ids[5:10], vals[5:10], dloss[5:10], tail=tail, temperature=T)
    assert torch.isnan(loss[:4]).all() and torch.isnan(g[:4]).all() and torch.isfinite(g[4]).all()


def test_no_list():
    z, _ = ref.random_logits(3, 100, F32, 1)
    ids = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    vals = torch.empty(3, 0, device="cuda")
    for tail in (False, True):
        loss, stats, g = lmh.lmhead_distill_fused(z, ids, vals, torch.ones(1, device="cuda"), tail=tail)
        assert (loss == 0).all() and (g == 0).all() and (stats == 0).all()
    z0 = torch.empty(0, 100, device="cuda")
    got = lmh.lmhead_distill_fused(z0, ids[:0], vals[:0], torch.ones(1, device="cuda"))
    assert [tuple(t.shape) for t in got] == [(0,), (0, 8), (0, 100)]


def test_pitched_lists_and_given_outputs():
    z, gen = ref.random_logits(6, 3000, F32, 1)
    ids = torch.stack([torch.randperm(3000, device="cuda", generator=gen)[:33] for _ in range(6)]).int()
    vals = torch.randn(6, 33, device="cuda", generator=gen).bfloat16()
    a = lmh.lmhead_distill_fwd(z, ids[:, 1:21], vals[:, 1:21])
    b = lmh.lmhead_distill_fwd(z, ids[:, 1:21].contiguous(), vals[:, 1:21].contiguous())
    outs = (torch.empty(6, device="cuda"), torch.empty(6, 8, device="cuda"))
    ws = torch.empty(lmh.lmhead_distill_workspace_bytes(6, 3000), dtype=torch.uint8, device="cuda")
    c = lmh.lmhead_distill_fwd(z, ids[:, 1:21], vals[:, 1:21], loss=outs[0], stats=outs[1], workspace=ws)
    for x, y, w, o in zip(a, b, c, outs):
        assert torch.equal(x, y) and w is o and torch.equal(x, w)
    none, stats = lmh.lmhead_distill_fwd(z, ids[:, 1:21], vals[:, 1:21], loss=False)
    assert none is None and torch.equal(stats, a[1])
    side = torch.cuda.Stream()
    up = torch.ones(1, device="cuda")
    want = lmh.lmhead_distill_fused(z, ids, vals, up)
    torch.cuda.synchronize()
    for st in (side, side.cuda_stream):
        got = lmh.lmhead_distill_fused(z, ids, vals, up, workspace=ws, stream=st)
        g = lmh.lmhead_distill_bwd(z, want[1], ids, vals, up, stream=st)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert torch.allclose(g, want[2], rtol=1e-5, atol=1e-7)


@pytest.mark.parametrize("tail", [False, True])
def test_rows_in_many_parts(tail):
    """Few long rows: parts and their merge, over a workspace of any contents."""
    n, V, k = 2, 1_200_003, 200
    for dtype in (F32, BF16):
        z, gen = ref.random_logits(n, V, dtype, 3)
        ids = torch.randint(0, V, (n, k), device="cuda", generator=gen).int()
        ids[0, 3] = ids[0, 190] = V - 1
        vals = torch.log_softmax(torch.randn(n, k, device="cuda", generator=gen), 1) - 0.3
        up = torch.ones(1, device="cuda")
        ws = torch.full((lmh.lmhead_distill_workspace_bytes(n, V),), 255, dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0
        want = ref.distill(z, ids, vals, tail, None, up)
        loss, stats, g = lmh.lmhead_distill_fused(z, ids, vals, up, tail=tail, workspace=ws, grad_dtype=F32)
        ref.assert_within(loss, want["loss"], want["tol_loss"], "loss")
        ref.assert_grad(g, want["dlogits"], want["tol_dlogits"], "dlogits")
        ws.fill_(255)
        again = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail, workspace=ws)
        assert torch.equal(again[0], loss) and torch.equal(again[1], stats)
        ids[1] = -1
        loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=tail, workspace=ws)
        assert torch.equal(loss[0], again[0][0]) and loss[1] == 0 and (stats[1] == 0).all()


def test_more_rows_than_one_launch_takes():
    """2^21 rows a launch."""
    n, V = 2 ** 21 + 5, 8
    gen = torch.Generator(device="cuda").manual_seed(4)
    z = torch.randn(n, V, device="cuda", generator=gen)
    ids = torch.randint(0, V, (n, 2), device="cuda", generator=gen).int()
    vals = torch.log_softmax(torch.randn(n, 2, device="cuda", generator=gen), 1) - 0.5
    T = 0.5 + torch.rand(n, device="cuda", generator=gen)
    up = torch.randn(n, device="cuda", generator=gen)
    loss, stats = lmh.lmhead_distill_fwd(z, ids, vals, tail=True, temperature=T)
    g = lmh.lmhead_distill_bwd(z, stats, ids, vals, up, tail=True, temperature=T)
    fused = lmh.lmhead_distill_fused(z, ids, vals, up, tail=True, temperature=T)
    want = ref.distill(z, ids, vals, True, T, up)
    for got_loss, got in ((loss, g), fused[::2]):
        ref.assert_within(got_loss, want["loss"], want["tol_loss"], "loss")
        ref.assert_grad(got, want["dlogits"], want["tol_dlogits"], "dlogits")


def test_offsets_past_32_bits():
    V, n, k = 131072, 16500, 3
    z = torch.zeros(n, V, dtype=BF16, device="cuda")
    z[n - 1, V - 1] = 4.0
    ids = torch.tensor([V - 1, 5, 77], dtype=torch.int32, device="cuda").expand(n, k).contiguous()
    vals = torch.tensor([-0.5, -2.0, -3.0], device="cuda").expand(n, k).contiguous()
    up = torch.ones(1, device="cuda")
    want = ref.distill(z[n - 2:], ids[n - 2:], vals[n - 2:], True, None, up)
    loss, stats, g = lmh.lmhead_distill_fused(z, ids, vals, up, tail=True, in_place=True)
    ref.assert_within(loss[n - 2:], want["loss"], want["tol_loss"], "loss")
    ref.assert_grad(g[n - 2:], want["dlogits"], want["tol_dlogits"], "dlogits")


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    n, V, k, eps = 3, 1031, 9, 1e-4
    z, gen = ref.random_logits(n, V, F32, 8, sigma=1.5)
    T = 0.7 + 0.6 * torch.rand(n, device="cuda", generator=gen)
    ids, vals = _lists(z, k, tail, F32, gen, ragged=False, T=T)
    up = torch.ones(1, device="cuda")
    _, _, got = lmh.lmhead_distill_fused(z, ids, vals, up, tail=tail, temperature=T)
    for j in {0, 3, 77, 1030, *ids[0].tolist()[:3], *ids[2].tolist()[:2]} - {-1}:
        hi, lo = z.double().clone(), z.double().clone()
        hi[:, j] += eps
        lo[:, j] -= eps
        diff = (ref.distill(hi, ids, vals, tail, T, up)["loss"] -
                ref.distill(lo, ids, vals, tail, T, up)["loss"]) / (2 * eps)
        assert torch.allclose(got[:, j].double(), diff, rtol=1e-5, atol=1e-6), j


def test_teacher_to_student_step_captured():
    """A teacher's logits to its alternatives, those to the student's loss and
    weight gradients, captured and replayed on other inputs."""
    M, K, V, k = 40, 128, 5008, 12
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    Wt = (0.2 * torch.randn(V, K, device="cuda", generator=gen)).bfloat16()
    W = (0.1 * torch.randn(V, K, device="cuda", generator=gen)).bfloat16()
    T = torch.full((1,), 1.5, device="cuda")
    up = torch.full((1,), 1.5 ** 2 / M, device="cuda")

    def step():
        zt = lmh.lmhead_logits(x, Wt, out_dtype="fp32")
        _, _, _, top_lp, top_tok, _ = lmh.lmhead_logprobs(zt, n_top=k, temperature=T, entropy=False)
        z = lmh.lmhead_logits(x, W, out_dtype="fp32")
        loss, _, dz = lmh.lmhead_distill_fused(z, top_tok, top_lp, up, tail=True, temperature=T, grad_dtype="bf16")
        return zt, z, top_tok, top_lp, loss, dz, lmh.lmhead_dgrad(dz, W, dx_dtype="fp32"), lmh.lmhead_wgrad(dz, x)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(torch.randn(M, K, device="cuda", generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), i
        _, z, tok, lp, loss, dz, _, _ = eager
        want = ref.distill(z, tok, lp, True, T, up)
        ref.assert_within(loss, want["loss"], want["tol_loss"], "loss")
        ref.assert_grad(dz, want["dlogits"], want["tol_dlogits"], "dlogits")
    # a student that is the teacher has nothing to learn from the full list
    zt = outs[0]
    _, _, _, lp, tok, _ = lmh.lmhead_logprobs(zt, n_top=64, temperature=T)
    loss, _, g = lmh.lmhead_distill_fused(zt, tok, lp, up, tail=True, temperature=T)
    assert loss.abs().max() < 1e-5 and g.abs().max() < 1e-5 * float(up)
