"""Beam selection where the scores leave the range of FP32, or lie at its ends.

The scores are FP64: a beam at the type's lowest value over a logit masked with
that value offers a candidate near -6.8e38, which is a better one than -inf.
Every result buffer is filled beforehand with values that no selection returns,
so a position that is not written shows.  The oracle is the definition in 64
bits, c = s + ((z - max) - log sum exp(z - max)), rounded to FP32 at the end
(below -FLT_MAX - half a step: -inf)."""
import numpy as np
import pytest
import torch

import lm_head_fp32_amd as lmh

pytestmark = pytest.mark.gpu

LOW = torch.finfo(torch.float32).min
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


def _rows(t):
    mult = 16 // t.element_size()
    ld = (t.shape[-1] + mult - 1) // mult * mult
    buf = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, : t.shape[-1]] = t
    return buf[:, : t.shape[-1]]


def _oracle(z, s, k, fin, eos):
    """Per request: the k first of (score, beam, token), FP64 scores."""
    B, W = s.shape
    z = z.double().cpu().numpy()
    V = z.shape[1]
    s = s.double().cpu().numpy()
    out = []
    for b in range(B):
        c = np.full((W, V), -np.inf)
        for w in range(W):
            if not -np.inf < s[b, w] < np.inf:
                continue
            row = z[b * W + w]
            m = row.max()
            if fin[b, w]:
                if 0 <= eos < V:
                    c[w, eos] = s[b, w]
            elif np.isfinite(m):
                c[w] = s[b, w] + ((row - m) - np.log(np.exp(row - m).sum()))
        beam, tok = np.divmod(np.arange(W * V), V)
        # ties: the lower beam, then the larger logit, then the lower token
        # (between candidates of -inf the position alone)
        logit = np.where(np.isneginf(c), 0.0, z[b * W:(b + 1) * W]).ravel()
        order = np.lexsort((tok, -logit, beam, -c.ravel()))[:k]
        out.append([(c.ravel()[i], int(beam[i]), int(tok[i])) for i in order])
    return out


def _check(z, s, k, fin=None, eos=-1):
    B, W = s.shape
    f = torch.zeros(B, W, dtype=torch.bool) if fin is None else fin
    want = _oracle(z, s, k, f.numpy(), eos)
    out = [torch.full((B, k), 12345.0, device="cuda"),
           torch.full((B, k), -77, dtype=torch.int32, device="cuda"),
           torch.full((B, k), -77, dtype=torch.int32, device="cuda"),
           torch.full((B, k), 7, dtype=torch.uint8, device="cuda")]
    lmh.lmhead_beam_select(_rows(z.cuda()), s.cuda(), n_out=k, finished=None if fin is None else fin.cuda(),
                           eos=eos, out_scores=out[0], out_parent=out[1], out_token=out[2],
                           out_finished=out[3])
    torch.cuda.synchronize()
    sc, par, tok, end = (t.cpu() for t in out)
    for b in range(B):
        assert list(zip(par[b].tolist(), tok[b].tolist())) == [q[1:] for q in want[b]], b
        for i, (c, w, v) in enumerate(want[b]):
            # FP32 rounding by half a step; the sums differ by 4e-9 at most
            with np.errstate(over="ignore"):
                r = float(np.float32(c))
            g = float(sc[b, i])
            assert g == r or abs(g - c) <= abs(c) * 2.0 ** -24 + 4e-9, (b, i, g, c)
            assert end[b, i] == int(bool(f[b, w]) or v == eos), (b, i)


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [4, 65, 5000])
def test_lowest_scores_over_lowest_masks(V, dtype):
    """Beams at finfo.min, one token of each row permitted, twice as many
    results as beams: the masked tokens come next, not what the buffers held."""
    low = torch.finfo(dtype).min
    z = torch.full((4, V), low, dtype=dtype)
    for w, j in enumerate((1, 3, 0, V - 1)):
        z[w, j] = 0.0
    for k in (1, 2, 4, 8):
        _check(z, torch.full((2, 2), LOW), k)
    _check(z, torch.tensor([[LOW, -3.0], [-1.5, LOW]]), 6)
    _check(z, torch.tensor([[LOW, -INF], [-INF, LOW]]), 5)
    _check(z, torch.full((1, 4), LOW), 12)
    # a beam that has ended beside them
    _check(z, torch.full((2, 2), LOW), 4, torch.tensor([[True, False], [False, True]]), 2)


@pytest.mark.parametrize("k", [1, 2, 3, 4])
def test_logits_at_both_ends(k):
    """Scores below the FP32 range from the logits alone; all of a row's
    candidates are asked for."""
    _check(torch.tensor([[3e38, -3e38, -3e38, -3e38]]), torch.zeros(1, 1), k)
    _check(torch.tensor([[-3e38, 3e38, -INF, -3.4e38]]), torch.zeros(1, 1), k)
    _check(torch.tensor([[-3e38, 3e38, -2e38, 3e38]]), torch.full((1, 1), -3e38), k)
    _check(torch.tensor([[LOW, LOW, LOW, LOW]]), torch.full((1, 1), LOW), k)


def test_below_the_range_comes_before_nothing():
    """A candidate below the FP32 range is better than one at -inf."""
    z = torch.full((2, 300), -INF)
    z[0, 5], z[0, 250], z[0, 7] = 0.0, LOW, LOW
    z[1, 290] = 1.0
    for k in (1, 2, 3, 4, 9):
        _check(z, torch.full((1, 2), LOW), k)
        _check(z, torch.tensor([[LOW, -2.0]]), k)


def test_many_below_the_range():
    """More of them than the merge ranks at once, and lists of several segments."""
    for W, V, k in ((1, 9000, 64), (33, 2100, 64), (3, 64, 40)):
        z = torch.full((2 * W, V), LOW)
        z[::2, 11] = 2.0
        _check(z, torch.full((2, W), LOW), k)


def test_constrained_search_with_finite_masks():
    """Masks of finfo.min step after step, 2 W results each, as a search that
    lets few tokens through runs; one beam ends on the way."""
    W, V = 2, 6
    s = torch.tensor([[0.0, LOW]])
    fin = torch.zeros(1, W, dtype=torch.bool)
    for step in range(4):
        z = torch.full((W, V), LOW)
        z[:, 3] = 0.5
        _check(z, s, 2 * W, fin, 3)
        sc, _, _, ended = lmh.lmhead_beam_select(_rows(z.cuda()), s.cuda(), n_out=2 * W, finished=fin.cuda(),
                                                 eos=3)
        s, fin = sc[:, :W].cpu().contiguous(), ended[:, :W].cpu().contiguous()


@pytest.mark.parametrize("W,B", [(1, 2 ** 23), (3, 2 ** 22 + 5)])
def test_as_many_requests_as_allowed(W, B):
    """More requests than one launch of the merge covers, in place; the best of
    one or two tokens per beam and the beams' ends."""
    g = torch.Generator(device="cuda").manual_seed(W)
    z = torch.zeros((B * W, 4), device="cuda")[:, :2]
    z[:, 1] = torch.where(torch.rand(B * W, device="cuda", generator=g) < 0.5, -2.0, 1.0)
    s = -torch.arange(B, device="cuda").remainder(1000)[:, None] - 8.0 * torch.rand(B, W, device="cuda", generator=g)
    fin = torch.rand(B, W, device="cuda", generator=g) < 0.25
    a, m = z.double(), z.double().amax(1, keepdim=True)
    c = ((a - m) - torch.log(torch.exp(a - m).sum(1, keepdim=True))).view(B, W, 2) + s.double()[:, :, None]
    held = torch.stack([torch.full_like(s.double(), -INF), s.double()], 2)  # eos is token 1
    c = torch.where(fin[:, :, None], held, c).view(B, 2 * W)
    best, at = torch.sort(c, dim=1, descending=True, stable=True)
    best, at = best[:, :W], at[:, :W].int()
    if W > 1:  # no two of a request's scores closer than the kernel's bound on them
        gap = best[:, :-1] - best[:, 1:]
        sure = (gap > 1e-8).all(1) & (c.sort(1, descending=True).values[:, W] < best[:, -1] - 1e-8)
    else:
        sure = torch.ones(B, dtype=torch.bool, device="cuda")
    assert sure.float().mean() > 0.99 and sure[-3:].any()
    ended = torch.gather(fin, 1, (at // 2).long()) | (at % 2 == 1)
    sc, par, tok, end = lmh.lmhead_beam_select(z, s, finished=fin, eos=1, out_scores=s, out_finished=fin)
    torch.cuda.synchronize()
    assert torch.equal(par[sure], (at // 2)[sure]) and torch.equal(tok[sure], (at % 2)[sure])
    assert torch.equal(end[sure], ended[sure])
    assert ((sc.double() - best).abs() <= best.abs() * 2.0 ** -24 + 4e-9)[torch.isfinite(best)].all()


def test_reorder_rows_of_more_than_31_bits():
    """Rows of 2 GiB and more that move whole, to other memory and in place."""
    T = 2 ** 31 + 4099
    st = torch.zeros((4, T), dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 1, 4097, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 4096, T - 1], device="cuda")
    marks = torch.arange(28, dtype=torch.uint8, device="cuda").view(4, 7) + 1
    st[:, at] = marks
    par = torch.tensor([[2, 0, 0, 3], [1, 3, 2, 0]], dtype=torch.int32, device="cuda")
    out = lmh.lmhead_beam_reorder(st, par[:1], out=torch.full_like(st, 99))
    assert torch.equal(out[:, at], marks[par[0].long()])
    assert int(out[:, :2 ** 20].sum()) == int(out[:, at[:3]].sum()) and not out[:, -4000:-3].any()
    del out
    lmh.lmhead_beam_reorder(st, par[1:])
    assert torch.equal(st[:, at], marks[par[1].long()])
    assert not st[:, 8192:2 ** 20].any() and not st[:, -4000:-3].any()
